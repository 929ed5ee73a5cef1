"""GPU: MXFP4 calls on tensors past 2^32 bytes and on more matrices than one line of a grid has tiles."""

from __future__ import annotations

import pytest
import torch

import mxfp4_helpers as M
import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV
from test_gpu_expert_mlp import check, gen

pytestmark = pytest.mark.gpu


def codes(*shape, seed=1):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen(seed))


def scales(*shape, seed=2):
    return torch.randint(116, 121, shape, dtype=torch.uint8, device=DEV, generator=gen(seed))


def test_quantize_and_back():
    rows, cols, tail = (1 << 17) + 3, 1 << 16, 259  # 2^33 values and more
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    for i in range(0, rows, 1 << 15):
        x[i:i + (1 << 15)].normal_(generator=gen(i))
    row, col = nv.mxfp4_quantize(x, columnwise=True)
    for lo in (0, rows - tail):
        want, wcol = nv.mxfp4_quantize(x[lo:lo + tail].contiguous(), columnwise=True)
        assert torch.equal(row.data[lo:lo + tail], want.data) and torch.equal(row.scales[:, lo:lo + tail], want.scales)
        if lo == 0:
            assert torch.equal(col.data[:, :128], wcol.data[:, :128]) and torch.equal(col.scales[:2], wcol.scales[:2])
    last = nv.mxfp4_quantize(x[1 << 17:].contiguous(), columnwise=True)[1]  # the last block of the columns: three rows
    assert torch.equal(col.data[:, -64:], last.data) and torch.equal(col.scales[-1:], last.scales)
    del x, col
    y = nv.mxfp4_dequantize(row)
    assert torch.equal(y[-tail:], nv.mxfp4_dequantize(nv.Mxfp4Tensor(row.data[-tail:].contiguous(), row.scales[:, -tail:].contiguous(), tail, cols)))


@pytest.mark.parametrize("block_2d", [False, True])
def test_more_matrices_than_one_grid_line_has_tiles(block_2d):
    batch = (1 << 24) + 3
    x = torch.randn((batch, 1, 1), device=DEV, generator=gen(2)).to(torch.bfloat16)
    row, col = nv.mxfp4_quantize(x, columnwise=True, block_2d=block_2d)
    want = nv.mxfp4_quantize(x[:, :, 0])[0]  # as rows of one matrix
    for q in (row, col):
        assert torch.equal(q.data[:, 0], want.data) and torch.equal(q.scales[:, 0, 0], want.scales[0])
        assert torch.equal(nv.mxfp4_dequantize(q)[:, 0], nv.mxfp4_dequantize(want))


def test_product_of_a_large_operand():
    m, k, tail = (1 << 17) + 5, 1 << 16, 100
    a = nv.Mxfp4Tensor(codes(m, k // 2), scales(k // 128, m, 4), m, k)
    b = nv.Mxfp4Tensor(codes(40, k // 2, seed=3), scales(k // 128, 40, 4, seed=4), 40, k)
    for p, q, t in ((a, b, False), (b, a, True)):
        d = nv.mxfp4_matmul(p, q, out_dtype=torch.float32)
        d = d.t() if t else d
        last = nv.Mxfp4Tensor(a.data[-tail:].contiguous(), a.scales[:, -tail:].contiguous(), tail, k)
        M.check_product(d[-tail:], M.values(last), M.values(b))


def test_large_results():
    m, n, k, tail = (1 << 16) + 130, 1 << 15, 128, 140
    a = nv.Mxfp4Tensor(codes(m, 64), scales(1, m, 4), m, k)
    b = nv.Mxfp4Tensor(codes(n, 64, seed=3), scales(1, n, 4, seed=4), n, k)
    d = nv.mxfp4_matmul(a, b)
    M.check_product(d[-tail:].contiguous(), M.values(a)[-tail:], M.values(b))


def test_grouped_products_with_large_weights():
    experts, n, k = 64, 8200, 1 << 14
    w = nv.Mxfp4Tensor(codes(experts, n, k // 2), scales(experts, k // 128, n, 4), n, k)
    ids = torch.arange(experts - 1, experts - 4, -1, dtype=torch.int32, device=DEV)[:, None]
    plan = nv.expert_sort(ids, experts, align=16)
    a = nv.Mxfp4Tensor(codes(plan.rows, k // 2, seed=5), scales(k // 128, plan.rows, 4, seed=6), plan.rows, k)
    d = nv.mxfp4_matmul_grouped(a, w, plan, out_dtype=torch.float32)
    va, off = M.values(a), plan.offsets.tolist()
    M.check_product(d[off[-2]:off[-1]], va[off[-2]:off[-1]], M.values(w, experts - 1))


def test_layer_with_large_weights():
    experts, cols, hidden = 64, 1 << 14, 4096 + 8
    kb1, kb2 = cols // 128, -(-hidden // 128)
    w1 = nv.Mxfp4Tensor(codes(experts, 2 * hidden, cols // 2), scales(experts, kb1, 2 * hidden, 4), 2 * hidden, cols)
    w2 = nv.Mxfp4Tensor(codes(experts, cols, kb2 * 64, seed=3), scales(experts, kb2, cols, 4, seed=4), cols, hidden)
    w2.data[:, :, hidden // 2:] = 0
    x = (torch.randn((2, cols), device=DEV, generator=gen(7)) / 64).bfloat16()
    ids = torch.tensor([[63], [62]], dtype=torch.int32, device=DEV)
    weights = torch.ones((2, 1), device=DEV)
    check(nv.expert_mlp(x, ids, weights, w1, w2), x, ids, weights, w1, w2, True)
