"""GPU: block-scaled FP8 products whose scales leave the middle of binary32's
range: what the definition gives is a normal number, zero or an infinity, and
so is the result, also where the product of two scales is out of range."""

from __future__ import annotations

import pytest
import torch

import expert_helpers as H
import fp8_helpers as F
import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

# one size for each kernel that the sizes choose between: few rows with one to eight shares of k, 64x64,
# 64x128, 128x128 and 256x256 tiles
SIZES = [(1, 40, 300), (16, 100, 900), (30, 70, 1600), (32, 65, 3200), (100, 77, 520), (1100, 1300, 260), (2100, 2052, 260), (3000, 2816, 260)]


# exponents of a's and of b's blocks: products from 2^-130 to 2^-90 whose scales multiply to denormals and
# to zero; scales at the ends of the range that meet in its middle; every block an exponent of its own
RANGES = [((-67, -63), (-67, -63)), ((-62, -58), (-62, -58)), ((-56, -50), (-56, -50)), ((-100, -96), (-22, -18)), ((110, 118), (-118, -110)), ((-110, -100), (100, 110)),
          ((60, 63), (60, 63)), ((-60, 60), (-60, 60)), ((-120, 118), (-120, 118))]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("b_2d,out", [(True, torch.bfloat16), (True, torch.float32), (False, torch.bfloat16), (False, torch.float32)])
def test_scales_far_from_one(m, n, k, b_2d, out):
    for i, (ra, rb) in enumerate(RANGES):
        a, b = F.operand(m, k, False, i, exponents=ra), F.operand(n, k, b_2d, 100 + i, exponents=rb)
        F.check_product(nv.fp8_matmul(a, b, out_dtype=out), F.values(a), F.values(b))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("b_2d", [True, False])
def test_zero_sums_of_large_operands_are_zero(m, n, k, b_2d):
    # scales of 2^100 each; the codes have no place in common in the first block, cancel in the second, and are
    # zero in the others: every sum is 0
    a, b = F.operand(m, k, False, 1), F.operand(n, k, b_2d, 2)
    for q, half in ((a, 0), (b, 1)):
        q.scales.fill_(2.0 ** 100)
        v = q.data.float()
        v[:, half:128:2] = 0
        v[:, 128:] = 0
        q.data.copy_(v.to(q.data.dtype))
    if k >= 256:
        va, vb = a.data.float(), b.data.float()
        va[:, 128:256], vb[:, 128:192], vb[:, 192:256] = 2, 3, -3
        a.data.copy_(va.to(a.data.dtype))
        b.data.copy_(vb.to(b.data.dtype))
    for out in (torch.bfloat16, torch.float32):
        assert torch.equal(nv.fp8_matmul(a, b, out_dtype=out), torch.zeros((m, n), dtype=out, device=DEV))


def test_values_near_1e_minus_20():
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.randn((200, 640), device=DEV, generator=g) * 1e-20
    w = torch.randn((300, 640), device=DEV, generator=g) * 1e-17
    for a, b in ((x, w), (w, x)):
        qa, qb = nv.fp8_quantize(a)[0], nv.fp8_quantize(b, block_2d=True)[0]
        F.check_product(nv.fp8_matmul(qa, qb, out_dtype=torch.float32), F.values(qa), F.values(qb))


@pytest.mark.parametrize("counts,n", [([3, 0, 20, 1], 70), ([100, 33, 300], 200), ([900, 1000, 1100], 4096)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_groups_with_scales_far_from_one(counts, n, out):
    k = 520
    plan = F.plan_of(counts, 16)
    off = H.i64(plan.offsets)
    for ra, rb in RANGES:
        a, b = F.operand(plan.rows, k, False, 1, exponents=ra), F.operand(n, k, True, 2, lead=(len(counts),), exponents=rb)
        d, va = nv.fp8_matmul_grouped(a, b, plan, out_dtype=out), F.values(a)
        for e in range(len(counts)):
            F.check_product(d[off[e]:off[e + 1]], va[off[e]:off[e + 1]], F.values(b, e))


@pytest.mark.parametrize("m,n", [(70, 60), (500, 500), (700, 1000), (1500, 1536)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_weight_gradients_with_scales_far_from_one(m, n, out):
    plan = F.plan_of([200, 0, 129, 1, 300], 128)
    off = H.i64(plan.offsets)
    for ra, rb in RANGES:
        a, b = F.operand(m, plan.rows, False, 1, exponents=ra), F.operand(n, plan.rows, False, 2, exponents=rb)
        d, va, vb = nv.fp8_matmul_grouped_k(a, b, plan, out_dtype=out), F.values(a), F.values(b)
        for e in range(5):
            F.check_product(d[e], va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]])
