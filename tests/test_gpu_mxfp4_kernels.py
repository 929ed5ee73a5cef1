"""GPU: every kernel that the sizes of an MXFP4 product choose between, at partial tiles and odd lengths; scales at the
ends of their range; the expert layer's kernels for many choices and for long rows."""

from __future__ import annotations

import pytest
import torch

import mxfp4_helpers as M
import nvfp4_block_scaled_05_amd as nv
from fp8_helpers import plan_of
from gpu_helpers import DEV
from test_gpu_expert_mlp import check, gen, layer

pytestmark = pytest.mark.gpu
OUT = [torch.bfloat16, torch.float32]

# few rows, with short and long k; 64x64, 64x128 and 128x128 tiles with k dealt out; 128x128; 256x256
FEW = [(1, 65, 2047), (16, 64, 15 * 128), (17, 63, 2048), (32, 130, 2049), (31, 1, 4100)]
TILES = [(100, 1000, 5), (65, 2000, 600), (1000, 2040, 385), (1024, 2048, 100), (2000, 2047, 999), (2040, 2048, 5), (2001, 4001, 1111), (2048, 4096, 128),
         (4001, 4095, 129), (4090, 4097, 77), (4096, 4096, 300)]


@pytest.mark.parametrize("m,n,k", FEW + TILES)
@pytest.mark.parametrize("out", OUT)
def test_partial_tiles(m, n, k, out):
    a, b = M.operand(m, k, m, exponents=(-3, 3)), M.operand(n, k, n, exponents=(-3, 3))
    M.check_product(nv.mxfp4_matmul(a, b, out_dtype=out), M.values(a), M.values(b))


# b's scales make up for a's
@pytest.mark.parametrize("m,n,k", [(1, 40, 300), (16, 100, 2300), (32, 65, 3200), (100, 77, 520), (1100, 1300, 260), (2000, 2040, 260), (2100, 4052, 260), (4000, 4096, 260)])
@pytest.mark.parametrize("exponents", [((110, 118), (-118, -110)), ((-100, -96), (70, 74)), ((-110, -100), (100, 110)), ((-30, -26), (-34, -30)), ((50, 53), (50, 53))])
def test_scales_far_from_one(m, n, k, exponents):
    a, b = M.operand(m, k, 1, exponents=exponents[0]), M.operand(n, k, 2, exponents=exponents[1])
    for out in OUT:
        M.check_product(nv.mxfp4_matmul(a, b, out_dtype=out), M.values(a), M.values(b))


def test_sums_past_the_largest_number_are_infinite():
    for m, n in ((8, 100), (100, 100), (2100, 4052), (4000, 4096)):
        a, b = M.operand(m, 256, 3), M.operand(n, 256, 4)
        for q in (a, b):
            q.data.fill_(0x77)  # sixes
            q.scales.fill_(200)
        assert bool((nv.mxfp4_matmul(a, b, out_dtype=torch.float32) == torch.inf).all())


GROUPS = [([64, 1, 65, 130], 1, 64, 300), ([63, 128, 129], 16, 200, 77), ([700, 1, 1000], 16, 1000, 385), ([1100, 1030], 1, 4100, 130), ([64] * 4, 16, 129, 128)]


@pytest.mark.parametrize("counts,align,n,k", GROUPS)
@pytest.mark.parametrize("out", OUT)
def test_groups(counts, align, n, k, out):
    plan = plan_of(counts, align)
    a, b = M.operand(plan.rows, k, 5, exponents=(-2, 2)), M.operand(n, k, 6, lead=(len(counts),), exponents=(-2, 2))
    d = nv.mxfp4_matmul_grouped(a, b, plan, out_dtype=out)
    va, off = M.values(a), plan.offsets.tolist()
    for e in range(len(counts)):
        M.check_product(d[off[e]:off[e + 1]], va[off[e]:off[e + 1]], M.values(b, e), f"group {e}")


@pytest.mark.parametrize("counts,m,n", [([130, 0, 1], 100, 70), ([128] * 8, 500, 1000), ([1, 300], 1000, 1001), ([700, 0, 129], 1500, 1536), ([256], 4090, 4097)])
def test_groups_along_k(counts, m, n):
    plan = plan_of(counts, 128)
    a, b = M.operand(m, plan.rows, 7, exponents=(-2, 2)), M.operand(n, plan.rows, 8, exponents=(-2, 2))
    d = nv.mxfp4_matmul_grouped_k(a, b, plan)
    va, vb, off = M.values(a), M.values(b), plan.offsets.tolist()
    for e in range(len(counts)):
        M.check_product(d[e], va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]], f"group {e}")


# long rows, whose tokens the registers hold in parts; many choices for few experts; both
LAYERS = [(3, 2, 4, 8200, 136), (2, 2, 4, 5300, 96), (3, 2, 4, 136, 4200), (1, 1, 2, 264, 8192), (40, 2, 2, 2056, 136), (40, 2, 2, 4104, 136), (70, 3, 4, 136, 2100),
          (33, 2, 2, 120, 4168), (30, 2, 2, 4100, 136), (512, 2, 3, 1000, 520), (1024, 1, 1, 72, 40), (300, 3, 20, 2049, 130), (13, 1, 1, 8192, 8192), (12, 1, 1, 256, 256)]


# rows of few blocks, which fewer waves share, with strips that end past the results
SHORT = [(100, 3, 64, 256, 1300), (100, 3, 64, 2100, 200), (500, 2, 64, 250, 1400), (500, 2, 64, 2100, 200), (64, 8, 64, 1000, 300), (40, 4, 128, 130, 2000),
         (90, 2, 64, 520, 700), (512, 2, 64, 400, 600), (5, 2, 8, 9, 40), (3, 2, 4, 7, 24), (20, 1, 1, 15, 9), (6, 2, 3, 127, 33)]


@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", LAYERS + SHORT)
@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [True, False])
def test_layers(tokens, topk, experts, cols, hidden, kind, gated):
    g = gen(tokens + hidden)
    x = torch.randn((tokens, cols), device=DEV, generator=g).bfloat16()
    ids = torch.randint(0, experts, (tokens, topk), dtype=torch.int32, device=DEV, generator=g)
    ids[tokens // 2, 0] = -1
    weights = torch.rand((tokens, topk), device=DEV, generator=g)
    w1, w2 = layer(kind, experts, cols, hidden, gated, cols)
    out = nv.expert_mlp(x, ids, weights, w1, w2, gated=gated)
    check(out, x, ids, weights, w1, w2, gated)
    for _ in range(3):
        assert torch.equal(nv.expert_mlp(x, ids, weights, w1, w2, gated=gated), out)


@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
def test_layer_of_infinities_and_of_none(kind):
    w1, w2 = layer(kind, 3, 264, 136, False, 9)
    x = torch.randn((6, 264), device=DEV, generator=gen(10)).bfloat16()
    ids = torch.tensor([[0], [1], [2], [0], [1], [-1]], dtype=torch.int32, device=DEV)
    weights = torch.ones((6, 1), device=DEV)
    x[1, 7], x[5, 3] = float("inf"), float("nan")
    x[2] = 0
    weights[3] = 0
    out = nv.expert_mlp(x, ids, weights, w1, w2, gated=False)
    assert not bool(torch.isfinite(out[1]).any())  # each row of w1 meets the infinity, or zero times it
    assert not bool(out[2].any()) and not bool(out[3].any()) and not bool(out[5].any())
    keep = [0, 4]
    clean = torch.where(torch.isfinite(x), x, 0)
    assert torch.equal(out[keep], nv.expert_mlp(clean, ids, weights, w1, w2, gated=False)[keep])
