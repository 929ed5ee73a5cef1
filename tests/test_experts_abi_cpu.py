"""Refusals of the expert-layer calls: every call here fails validation, so
nothing reaches a GPU."""

from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nvfp4.h")
P = 0x100000  # a fake, aligned device address


def q(data=P, scales=P):
    return nv.nvfp4_fp8_t(data, scales)


def sort(ids=P, id_bytes=4, tokens=8, topk=2, experts=4, align=16, rows=64, slot_rows=P, row_slots=P, offsets=P, counts=P, ws=None):
    return nv.load().nvfp4_expert_sort(ids, id_bytes, tokens, topk, experts, align, rows, slot_rows, row_slots, offsets, counts, ws, None)


@pytest.mark.parametrize("case,expected", [
    (dict(tokens=-1), nv.NVFP4_ERR_SHAPE), (dict(topk=0), nv.NVFP4_ERR_SHAPE), (dict(tokens=1 << 30, topk=2), nv.NVFP4_ERR_SHAPE),
    (dict(experts=0), nv.NVFP4_ERR_SHAPE), (dict(experts=257), nv.NVFP4_ERR_SHAPE), (dict(align=0), nv.NVFP4_ERR_UNSUPPORTED),
    (dict(align=24), nv.NVFP4_ERR_UNSUPPORTED), (dict(align=256), nv.NVFP4_ERR_UNSUPPORTED), (dict(id_bytes=2), nv.NVFP4_ERR_UNSUPPORTED),
    (dict(rows=63), nv.NVFP4_ERR_SHAPE), (dict(rows=1 << 31), nv.NVFP4_ERR_SHAPE), (dict(ids=None), nv.NVFP4_ERR_NULL),
    (dict(id_bytes=8, ids=P + 4), nv.NVFP4_ERR_ALIGN), (dict(offsets=None), nv.NVFP4_ERR_NULL), (dict(counts=None), nv.NVFP4_ERR_NULL),
    (dict(row_slots=None), nv.NVFP4_ERR_NULL), (dict(slot_rows=P + 2), nv.NVFP4_ERR_ALIGN),
    (dict(tokens=5000, rows=20000), nv.NVFP4_ERR_NULL),  # over 4096 slots: the workspace is missing
])
def test_sort_refuses(case, expected):
    assert sort(**case) == expected
    assert nv.nvfp4_last_error() != ""


def test_sizes():
    lib = nv.load()
    assert lib.nvfp4_expert_rows(64, 8, 64, 16) == 512 + 64 * 15
    assert lib.nvfp4_expert_rows(1, 2, 64, 128) == 256 and lib.nvfp4_expert_rows(10, 1, 3, 1) == 10
    assert lib.nvfp4_expert_rows(0, 8, 64, 16) == 0 and lib.nvfp4_expert_rows(8, 2, 4, 3) == 0
    assert lib.nvfp4_expert_sort_workspace_bytes(512, 8, 64) == 0
    assert 0 < lib.nvfp4_expert_sort_workspace_bytes(513, 8, 64) <= 256 * 64 * 4
    assert lib.nvfp4_expert_sort_workspace_bytes(1 << 27, 8, 256) <= 256 * 256 * 4
    assert [nv.nvfp4_fp8_pitch(k) for k in (-1, 0, 1, 128, 129)] == [0, 0, 128, 128, 256]


def test_row_moves_refuse():
    lib = nv.load()
    gather = lambda x=P, dt=0, t=8, k=2, c=64, s=P, m=P, r=32, y=P: lib.nvfp4_expert_gather(x, dt, t, k, c, s, m, r, y, None)  # noqa: E731
    assert gather(dt=2) == nv.NVFP4_ERR_UNSUPPORTED
    assert gather(t=-1) == gather(k=0) == gather(c=-1) == gather(r=-1) == gather(r=1 << 31) == nv.NVFP4_ERR_SHAPE
    assert gather(x=None) == gather(m=None) == gather(s=None) == gather(y=None) == nv.NVFP4_ERR_NULL
    assert gather(x=P + 8) == gather(y=P + 8) == gather(m=P + 2) == nv.NVFP4_ERR_ALIGN
    assert gather(r=0, x=None, s=None, m=None, y=None) == nv.NVFP4_OK
    combine = lambda y=P, dt=0, t=8, k=2, c=64, m=P, r=32, w=P, o=P: lib.nvfp4_expert_combine(y, dt, t, k, c, m, r, w, o, None)  # noqa: E731
    assert combine(dt=-1) == nv.NVFP4_ERR_UNSUPPORTED
    assert combine(y=None) == combine(m=None) == combine(o=None) == nv.NVFP4_ERR_NULL
    assert combine(w=P + 1) == combine(o=P + 4) == nv.NVFP4_ERR_ALIGN
    assert combine(t=1 << 29, k=1, c=1 << 30) == nv.NVFP4_ERR_SHAPE
    assert combine(t=0, y=None, m=None, w=None, o=None) == nv.NVFP4_OK

    def grad(g=P, y=P, dt=0, t=8, k=2, c=64, a=P, b=P, r=32, w=P, dy=P, dw=P):
        return lib.nvfp4_expert_combine_grad(g, y, dt, t, k, c, a, b, r, w, dy, dw, None)

    for name in ("g", "y", "a", "b", "w", "dy", "dw"):
        assert grad(**{name: None}) == nv.NVFP4_ERR_NULL, name
        assert grad(**{name: P + 2}) == nv.NVFP4_ERR_ALIGN, name
    assert grad(t=0, r=0, g=None, y=None, a=None, b=None, w=None, dy=None, dw=None) == nv.NVFP4_OK


def test_quantize_refuses():
    lib = nv.load()
    none = object()

    def call(x=P, dt=0, batch=1, rows=64, cols=64, slots=None, tokens=0, topk=1, row=none, col=None):
        row = q() if row is none else row
        return lib.nvfp4_fp8_quantize(x, dt, batch, rows, cols, slots, tokens, topk, 0, row, col, None)

    assert call(dt=5) == nv.NVFP4_ERR_UNSUPPORTED
    assert call(batch=-1) == call(rows=-1) == call(cols=-1) == call(rows=1 << 31) == call(cols=1 << 31) == nv.NVFP4_ERR_SHAPE
    assert call(batch=1 << 20, rows=1 << 13, cols=1 << 13) == nv.NVFP4_ERR_SHAPE
    assert call(row=None) == call(x=None) == call(row=q(data=None)) == call(row=q(scales=None)) == nv.NVFP4_ERR_NULL
    assert call(x=P + 8) == call(row=q(data=P + 8)) == call(row=None, col=q(scales=P + 2)) == nv.NVFP4_ERR_ALIGN
    assert call(slots=P, batch=2, tokens=8) == nv.NVFP4_ERR_UNSUPPORTED
    assert call(slots=P + 2, tokens=8) == nv.NVFP4_ERR_ALIGN
    assert call(slots=P, tokens=8, topk=0) == call(slots=P, tokens=-1) == nv.NVFP4_ERR_SHAPE
    assert call(rows=0, x=None, row=q(None, None)) == nv.NVFP4_OK


def test_products_refuse():
    lib = nv.load()

    def dense(a=None, b=None, m=64, n=64, k=64, d=P, dt=0):
        return lib.nvfp4_fp8_matmul(a or q(), b or q(), m, n, k, 1, d, dt, None)

    def grouped(f, a=None, b=None, off=P, g=4, rows=64, n=64, k=64, d=P, dt=0):
        return f(a or q(), b or q(), off, g, rows, n, k, d, dt, None)

    assert dense(dt=3) == nv.NVFP4_ERR_UNSUPPORTED
    assert dense(m=-1) == dense(n=1 << 31) == dense(k=1 << 23) == dense(m=1 << 30, n=1 << 30) == nv.NVFP4_ERR_SHAPE
    assert dense(a=q(data=None)) == dense(b=q(scales=None)) == dense(d=None) == nv.NVFP4_ERR_NULL
    assert dense(a=q(data=P + 4)) == dense(b=q(scales=P + 2)) == dense(d=P + 8) == nv.NVFP4_ERR_ALIGN
    assert lib.nvfp4_fp8_matmul(None, q(), 1, 1, 1, 0, P, 0, None) == nv.NVFP4_ERR_NULL
    assert dense(m=0, a=q(None, None), b=q(None, None), d=None) == nv.NVFP4_OK
    for f in (lib.nvfp4_fp8_matmul_grouped, lib.nvfp4_fp8_matmul_grouped_k):
        assert grouped(f, g=0) == grouped(f, g=257) == grouped(f, k=1 << 23) == nv.NVFP4_ERR_SHAPE
        assert grouped(f, off=None) == nv.NVFP4_ERR_NULL
        assert grouped(f, off=P + 2) == nv.NVFP4_ERR_ALIGN
        assert nv.nvfp4_last_error() != ""


def test_fp8_struct_matches_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "nvfp4.h"\nint main(void) { printf("%zu %zu %zu\\n", '
                   'sizeof(nvfp4_fp8_t), offsetof(nvfp4_fp8_t, data), offsetof(nvfp4_fp8_t, scales)); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    size, data, scales = map(int, subprocess.check_output([str(exe)]).split())
    T = nv.nvfp4_fp8_t
    assert (ctypes.sizeof(T), T.data.offset, T.scales.offset) == (size, data, scales)


def test_binding_refuses_host_tensors():
    ids = torch.zeros((4, 2), dtype=torch.int32)
    x = torch.zeros((4, 64))
    plan = nv.ExpertPlan(ids, torch.zeros(8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 128)
    f = nv.Fp8Tensor(torch.zeros((4, 128), dtype=torch.float8_e4m3fn), torch.zeros((1, 4)), 4, 64)
    for call in (lambda: nv.expert_sort(ids, 2), lambda: nv.expert_gather(x, plan), lambda: nv.expert_combine(x, plan),
                 lambda: nv.expert_combine_grad(x, x, plan, x), lambda: nv.fp8_quantize(x), lambda: nv.fp8_matmul(f, f),
                 lambda: nv.fp8_matmul_grouped(f, f, plan), lambda: nv.fp8_matmul_grouped_k(f, f, plan)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
