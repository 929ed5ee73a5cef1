"""Refusals of the MXFP4 calls and of the expert layer for a few tokens: every
call here fails validation, or has nothing to do, so nothing reaches a GPU."""

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
    return nv.nvfp4_mxfp4_t(data, scales)


def test_quantize_refuses():
    lib = nv.load()
    none = object()

    def call(x=P, dt=0, batch=1, rows=64, cols=64, slots=None, tokens=0, topk=1, row=none, col=None):
        row = q() if row is none else row
        return lib.nvfp4_mxfp4_quantize(x, dt, batch, rows, cols, slots, tokens, topk, 0, row, col, None)

    assert call(dt=5) == nv.NVFP4_ERR_UNSUPPORTED
    assert call(batch=-1) == call(rows=-1) == call(cols=-1) == call(rows=1 << 31) == call(cols=1 << 31) == nv.NVFP4_ERR_SHAPE
    assert call(batch=1 << 20, rows=1 << 13, cols=1 << 13) == nv.NVFP4_ERR_SHAPE
    assert call(row=None) == call(x=None) == call(row=q(data=None)) == call(row=q(scales=None)) == nv.NVFP4_ERR_NULL
    assert call(x=P + 8) == call(row=q(data=P + 8)) == call(row=None, col=q(scales=P + 2)) == nv.NVFP4_ERR_ALIGN
    assert call(slots=P, batch=2, tokens=8) == nv.NVFP4_ERR_UNSUPPORTED
    assert call(slots=P + 2, tokens=8) == nv.NVFP4_ERR_ALIGN
    assert call(slots=P, tokens=8, topk=0) == call(slots=P, tokens=-1) == nv.NVFP4_ERR_SHAPE
    assert call(rows=0, x=None, row=q(None, None)) == nv.NVFP4_OK
    assert nv.nvfp4_last_error() != ""


def test_dequantize_refuses():
    lib = nv.load()
    call = lambda t=None, batch=1, n=64, k=64, y=P, dt=0: lib.nvfp4_mxfp4_dequantize(t or q(), batch, n, k, y, dt, None)  # noqa: E731
    assert call(dt=2) == nv.NVFP4_ERR_UNSUPPORTED
    assert call(batch=-1) == call(n=-1) == call(k=1 << 31) == call(batch=1 << 20, n=1 << 13, k=1 << 13) == nv.NVFP4_ERR_SHAPE
    assert call(t=q(data=None)) == call(t=q(scales=None)) == call(y=None) == nv.NVFP4_ERR_NULL
    assert lib.nvfp4_mxfp4_dequantize(None, 1, 64, 64, P, 0, None) == nv.NVFP4_ERR_NULL
    assert call(t=q(data=P + 8)) == call(t=q(scales=P + 1)) == call(y=P + 4) == nv.NVFP4_ERR_ALIGN
    assert call(n=0, t=q(None, None), y=None) == call(batch=0, t=q(None, None), y=None) == nv.NVFP4_OK


def test_products_refuse():
    lib = nv.load()

    def dense(a=None, b=None, m=64, n=64, k=64, d=P, dt=0):
        return lib.nvfp4_mxfp4_matmul(a or q(), b or q(), m, n, k, d, dt, None)

    def grouped(f, a=None, b=None, off=P, g=4, rows=64, n=64, k=64, d=P, dt=0):
        return f(a or q(), b or q(), off, g, rows, n, k, d, dt, None)

    assert dense(dt=3) == nv.NVFP4_ERR_UNSUPPORTED
    assert dense(m=-1) == dense(n=1 << 31) == dense(k=1 << 23) == dense(m=1 << 30, n=1 << 30) == nv.NVFP4_ERR_SHAPE
    assert dense(a=q(data=None)) == dense(b=q(scales=None)) == dense(d=None) == nv.NVFP4_ERR_NULL
    assert dense(a=q(data=P + 4)) == dense(b=q(scales=P + 2)) == dense(d=P + 8) == nv.NVFP4_ERR_ALIGN
    assert lib.nvfp4_mxfp4_matmul(None, q(), 1, 1, 1, P, 0, None) == nv.NVFP4_ERR_NULL
    assert dense(m=0, a=q(None, None), b=q(None, None), d=None) == nv.NVFP4_OK
    for f in (lib.nvfp4_mxfp4_matmul_grouped, lib.nvfp4_mxfp4_matmul_grouped_k):
        assert grouped(f, g=0) == grouped(f, g=257) == grouped(f, k=1 << 23) == nv.NVFP4_ERR_SHAPE
        assert grouped(f, off=None) == nv.NVFP4_ERR_NULL
        assert grouped(f, off=P + 2) == nv.NVFP4_ERR_ALIGN
        assert nv.nvfp4_last_error() != ""


@pytest.mark.parametrize("m,n,k", [((1 << 31) - 1, 1, 1), ((1 << 31) - 1, 1, 0), (1, (1 << 31) - 1, 1), (32, (1 << 31) - 1, 26 * 128)])
def test_products_of_too_many_threads_are_refused(m, n, k):
    assert nv.load().nvfp4_mxfp4_matmul(q(), q(), m, n, k, P, nv.NVFP4_IN_BF16, None) == nv.NVFP4_ERR_SHAPE
    assert "too large for one launch" in nv.nvfp4_last_error()


@pytest.mark.parametrize("fp8", [False, True])
def test_expert_mlp_refuses(fp8):
    lib = nv.load()
    f = lib.nvfp4_expert_mlp_fp8 if fp8 else lib.nvfp4_expert_mlp_mxfp4
    w = (lambda data=P, scales=P: nv.nvfp4_fp8_t(data, scales)) if fp8 else q

    def call(x=P, tokens=8, cols=64, ids=P, id_bytes=4, weights=P, topk=2, experts=4, w1=None, w2=None, hidden=64, ws=P, out=P):
        return f(x, tokens, cols, ids, id_bytes, weights, topk, experts, w1 or w(), w2 or w(), hidden, 1, ws, out, None)

    assert call(tokens=-1) == call(topk=0) == call(experts=0) == call(experts=257) == call(tokens=513) == nv.NVFP4_ERR_SHAPE
    assert call(cols=0) == call(cols=1 << 23) == call(hidden=0) == call(hidden=1 << 23) == nv.NVFP4_ERR_SHAPE
    assert call(id_bytes=2) == nv.NVFP4_ERR_UNSUPPORTED
    assert call(x=None) == call(ids=None) == call(weights=None) == call(ws=None) == call(out=None) == nv.NVFP4_ERR_NULL
    assert call(w1=w(data=None)) == call(w2=w(scales=None)) == nv.NVFP4_ERR_NULL
    assert call(x=P + 8) == call(ids=P + 4, id_bytes=8) == call(weights=P + 2) == call(ws=P + 4) == call(out=P + 8) == nv.NVFP4_ERR_ALIGN
    assert call(w1=w(data=P + 8)) == call(w2=w(scales=P + 2)) == nv.NVFP4_ERR_ALIGN
    assert f(P, 8, 64, P, 4, P, 2, 4, None, w(), 64, 1, P, P, None) == nv.NVFP4_ERR_NULL
    assert call(tokens=0, x=None, ids=None, weights=None, w1=w(None, None), w2=w(None, None), ws=None, out=None) == nv.NVFP4_OK


def test_expert_mlp_workspace():
    size = nv.load().nvfp4_expert_mlp_workspace_bytes
    assert size(0, 2, 64, 64) % 16 == 0 and size(0, 2, 64, 64) > 0
    assert size(64, 8, 4096, 2048) - size(0, 8, 4096, 2048) == 512 * 4 * (2048 + 4096)
    assert size(3, 1, 65, 129) - size(0, 1, 65, 129) == 3 * 4 * (256 + 128)
    assert size(513, 2, 64, 64) == size(1, 1, 64, 0) == size(1, 1, 0, 64) == size(-1, 1, 64, 64) == size(1, 0, 64, 64) == 0


def test_struct_matches_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "nvfp4.h"\nint main(void) { printf("%zu %zu %zu %d\\n", sizeof(nvfp4_mxfp4_t), '
                   'offsetof(nvfp4_mxfp4_t, data), offsetof(nvfp4_mxfp4_t, scales), NVFP4_EXPERT_MLP_MAX_SLOTS); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    T = nv.nvfp4_mxfp4_t
    assert (ctypes.sizeof(T), T.data.offset, T.scales.offset, nv.NVFP4_EXPERT_MLP_MAX_SLOTS) == tuple(map(int, subprocess.check_output([str(exe)]).split()))


def test_binding_refuses_host_tensors():
    x, ids = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32)
    plan = nv.ExpertPlan(ids, torch.zeros(8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 128)
    t = nv.Mxfp4Tensor(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 4, 4), dtype=torch.uint8), 4, 64)
    for call in (lambda: nv.mxfp4_quantize(x), lambda: nv.mxfp4_dequantize(t), lambda: nv.mxfp4_matmul(t, t), lambda: nv.mxfp4_matmul_grouped(t, t, plan),
                 lambda: nv.mxfp4_matmul_grouped_k(t, t, plan), lambda: nv.expert_mlp(x, ids, torch.zeros((4, 2)), t, t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
