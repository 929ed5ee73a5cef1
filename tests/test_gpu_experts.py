"""GPU: tokens sorted by expert and back, and the gradients of both, against
plain 64-bit forms."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import expert_helpers as H
import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def make_ids(tokens, topk, experts, seed=0, drop=0.1, dtype=torch.int32):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((tokens, experts)) + 0.3 * rng.random(experts), axis=1)[:, :topk] if experts >= topk else \
        rng.integers(0, experts, (tokens, topk))
    ids = np.where(rng.random((tokens, topk)) < drop, rng.choice([-1, experts, 1 << 30, -(1 << 31)], (tokens, topk)), ids)
    return torch.from_numpy(np.ascontiguousarray(ids)).to(dtype).to(DEV)


def check_plan(ids, experts, align, rows=None):
    plan = nv.expert_sort(ids, experts, align=align, rows=rows)
    n = plan.rows
    assert rows is not None or n == H.capacity(ids.numel(), experts, align)
    want = H.sort(H.i64(ids), experts, align, n)
    for got, ref, name in zip((plan.slot_rows, plan.row_slots, plan.offsets, plan.counts), want,
                              ("slot_rows", "row_slots", "offsets", "counts")):
        assert got.dtype == torch.int32
        assert np.array_equal(H.i64(got), ref), name
    return plan


@pytest.mark.parametrize("tokens,topk,experts,align", [
    (1, 1, 1, 1), (1, 8, 8, 16), (64, 8, 64, 16), (63, 3, 7, 128), (512, 8, 256, 128), (513, 8, 255, 2),
    (1000, 4, 60, 16), (4097, 1, 5, 64), (8192, 8, 64, 128), (5000, 5, 256, 1)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(tokens, topk, experts, align, dtype):
    check_plan(make_ids(tokens, topk, experts, seed=tokens, dtype=dtype), experts, align)


def test_sort_int64_ids_that_differ_above_32_bits_are_dropped():
    ids = torch.tensor([[1 << 32, 0], [1, (1 << 40) + 1], [-(1 << 32), 1]], dtype=torch.int64, device=DEV)
    plan = check_plan(ids, 2, 16)
    assert H.i64(plan.counts).tolist() == [1, 2]


@pytest.mark.parametrize("tokens,topk", [(40, 3), (3000, 4)])
def test_sort_extremes(tokens, topk):
    everything = torch.full((tokens, topk), 2, dtype=torch.int32, device=DEV)
    check_plan(everything, 5, 128)                                              # one expert has them all
    check_plan(torch.full_like(everything, -1), 5, 128)                         # nobody has any
    check_plan(everything, 5, 16, rows=H.capacity(tokens * topk, 5, 16) + 77)   # more rows than needed


def test_sort_without_tokens():
    plan = check_plan(torch.empty((0, 4), dtype=torch.int32, device=DEV), 3, 16, rows=20)
    assert H.i64(plan.offsets).tolist() == [0, 0, 0, 0]


def test_sort_of_chunks_longer_than_a_tile():
    # over 256 * 4096 slots: a workgroup's chunk takes several tiles
    check_plan(torch.randint(-1, 37, (1100003, 1), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(1)), 37, 128)


def inputs(plan, cols, dtype, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn((plan.tokens, cols), device=DEV, generator=g).to(dtype)
    y = torch.randn((plan.rows, cols), device=DEV, generator=g).to(dtype)
    y[plan.row_slots < 0] = float("nan")  # padding is never read
    w = torch.rand((plan.tokens, plan.topk), device=DEV, generator=g)
    return x, y, w


SHAPES = [(1, 1, 2, 8, 1), (5, 3, 4, 1, 16), (64, 8, 64, 4096, 16), (33, 5, 7, 517, 128), (130, 2, 3, 1030, 64),
          (257, 8, 16, 100, 128), (40, 9, 32, 2049, 2)]


@pytest.mark.parametrize("tokens,topk,experts,cols,align", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gather_and_its_gradient(tokens, topk, experts, cols, align, dtype):
    plan = nv.expert_sort(make_ids(tokens, topk, experts, seed=cols), experts, align=align)
    x, dy, _ = inputs(plan, cols, dtype, seed=tokens)
    slots = H.i64(plan.row_slots)
    want = np.where((slots >= 0)[:, None], H.f64(x)[np.maximum(slots, 0) // topk], 0.0)
    assert np.array_equal(H.f64(nv.expert_gather(x, plan)), want)
    total, mag = H.combine(H.f64(dy), H.i64(plan.slot_rows), np.ones((tokens, topk)))
    H.close(nv.expert_gather_grad(dy, plan), total, mag * topk * 2.0 ** -24, "dx")


@pytest.mark.parametrize("tokens,topk,experts,cols,align", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine_and_its_gradients(tokens, topk, experts, cols, align, dtype):
    plan = nv.expert_sort(make_ids(tokens, topk, experts, seed=cols + 1), experts, align=align)
    dout, y, w = inputs(plan, cols, dtype, seed=tokens)
    rows, slots = H.i64(plan.slot_rows), H.i64(plan.row_slots)
    total, mag = H.combine(H.f64(y), rows, H.f64(w))
    H.close(nv.expert_combine(y, plan, w), total, mag * topk * 2.0 ** -24, "out")
    dy, dw = nv.expert_combine_grad(dout, y, plan, w)
    at = np.maximum(slots, 0)
    want = np.where((slots >= 0)[:, None], H.f64(dout)[at // topk] * H.f64(w).reshape(-1)[at][:, None], 0.0)
    H.close(dy, want, np.abs(want) * 2.0 ** -24, "dy")
    term = H.f64(dout)[:, None] * np.where((rows >= 0)[..., None], H.f64(y)[np.maximum(rows, 0)], 0.0)
    H.close(dw, term.sum(-1), np.abs(term).sum(-1) * cols * 2.0 ** -24, "dweights")


def test_combine_gradients_against_differences():
    # out is linear in y and in the weights, so a difference quotient is exact but for rounding
    plan = nv.expert_sort(make_ids(9, 3, 4, seed=5), 4, align=16)
    dout, y, w = inputs(plan, 40, torch.float32, seed=9)
    y = torch.nan_to_num(y)
    dy, dw = nv.expert_combine_grad(dout, y, plan, w)
    g = torch.Generator(DEV).manual_seed(3)
    for step_y, step_w in ((torch.randn(y.shape, device=DEV, generator=g), torch.zeros_like(w)),
                           (torch.zeros_like(y), torch.randn(w.shape, device=DEV, generator=g))):
        up, down = nv.expert_combine(y + step_y, plan, w + step_w), nv.expert_combine(y - step_y, plan, w - step_w)
        slope = ((up - down).double() * dout.double()).sum() / 2
        want = (dy.double() * step_y.double()).sum() + (dw.double() * step_w.double()).sum()
        scale = (dout.double().abs() * (up.double().abs() + down.double().abs())).sum()
        assert abs(float(slope - want)) <= float(scale) * 8 * 2.0 ** -24


def test_non_finite_rows_reach_only_their_tokens():
    ids = torch.tensor([[0, 1], [1, 0], [1, -1]], dtype=torch.int32, device=DEV)
    plan = nv.expert_sort(ids, 2, align=16)
    y = torch.ones((plan.rows, 24), device=DEV)
    y[int(plan.slot_rows[1, 0])] = float("inf")
    out = nv.expert_combine(y, plan, torch.ones((3, 2), device=DEV))
    assert torch.equal(out[0], torch.full((24,), 2.0, device=DEV)) and torch.equal(out[2], torch.ones(24, device=DEV))
    assert bool(torch.isinf(out[1]).all())


def test_rows_past_32_bits():
    # the sorted matrix has more than 2^32 bytes and 2^31 elements
    tokens, topk, cols = 34000, 8, 8192
    ids = torch.randint(0, 16, (tokens, topk), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    plan = nv.expert_sort(ids, 16, align=128)
    x = torch.randn((tokens, cols), device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(torch.bfloat16)
    y = nv.expert_gather(x, plan)
    assert y.numel() > 1 << 31
    last = plan.row_slots.long()
    for r in (0, plan.rows // 2, int((last >= 0).nonzero()[-1])):
        s = int(last[r])
        assert torch.equal(y[r], x[s // topk] if s >= 0 else torch.zeros_like(y[r]))
    out = nv.expert_combine(y, plan, torch.full((tokens, topk), 0.125, device=DEV))
    assert torch.equal(out, x)  # eighths of eight equal rows: every step is exact


def test_calls_on_another_stream_and_in_a_graph():
    ids = make_ids(64, 4, 8, seed=11)
    plan = nv.expert_sort(ids, 8, align=16)
    x, y, w = inputs(plan, 264, torch.bfloat16, seed=4)
    want = (nv.expert_gather(x, plan), nv.expert_combine(y, plan, w), *nv.expert_combine_grad(x, y, plan, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p2 = nv.expert_sort(ids, 8, align=16, stream=side)
    got = (nv.expert_gather(x, p2, stream=side), nv.expert_combine(y, p2, w, stream=side),
           *nv.expert_combine_grad(x, y, p2, w, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def step():
        p = nv.expert_sort(ids, 8, align=16)
        return (nv.expert_gather(x, p), nv.expert_combine(y, p, w), *nv.expert_combine_grad(x, y, p, w))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        ids.copy_(make_ids(64, 4, 8, seed=20 + k))
        graph.replay()
        torch.cuda.synchronize()
        p = nv.expert_sort(ids, 8, align=16)
        # rows of y that the new plan uses may have been padding before: NaN in both
        for a, b in zip(out, step()):
            assert torch.equal(torch.nan_to_num(a.float(), nan=-1e30), torch.nan_to_num(b.float(), nan=-1e30))
        assert int(p.counts.sum()) <= ids.numel()


def test_sorted_rows_are_the_groups_of_a_grouped_quantize():
    ids = make_ids(300, 4, 6, seed=8)
    plan = nv.expert_sort(ids, 6, align=16)
    x, _, _ = inputs(plan, 256, torch.bfloat16, seed=5)
    rows = int(plan.offsets[-1])
    group_rows = (plan.offsets[1:] - plan.offsets[:-1]).tolist()
    y = nv.expert_gather(x, plan)[:rows]
    row, _ = nv.quantize_grouped(y, group_rows, columnwise=False)
    at = 0
    for g, n in enumerate(group_rows):
        if n:
            one, _ = nv.quantize(y[at:at + n], columnwise=False)
            assert torch.equal(row.data.reshape(rows, -1)[at:at + n], one.data)
            assert float(row.amax[g]) == float(one.amax[0])
        at += n
