"""GPU: every kernel that the sizes of a product choose between, with both
forms of b's scales and both output types, against the product in 64 bits."""

from __future__ import annotations

import pytest
import torch

import expert_helpers as H
import fp8_helpers as F
import nvfp4_block_scaled_05_amd as nv

pytestmark = pytest.mark.gpu


OUT = [torch.bfloat16, torch.float32]

# few rows: one, two, four and eight waves share the blocks along k (up to 5, 11, 23 and more of them), with a share
# that ends in a part of what a wave asks for at once
ROWS = [(1, 100, 5 * 128), (32, 31, 3 * 128 + 1), (1, 100, 6 * 128), (16, 129, 7 * 128 - 3), (17, 64, 11 * 128), (32, 300, 9 * 128),
        (1, 70, 12 * 128), (16, 100, 13 * 128), (17, 33, 23 * 128 - 100), (31, 260, 16 * 128), (5, 64, 26 * 128), (32, 96, 41 * 128)]


@pytest.mark.parametrize("m,n,k", ROWS)
@pytest.mark.parametrize("b_2d", [True, False])
@pytest.mark.parametrize("out", OUT)
def test_few_rows(m, n, k, b_2d, out):
    a, b = F.operand(m, k, False, m + k), F.operand(n, k, b_2d, n)
    F.check_product(nv.fp8_matmul(a, b, out_dtype=out), F.values(a), F.values(b))


# 64x64 tiles with four shares of k, 64x128 with two, 128x128, 256x256 (two sizes of each: whole tiles and parts)
TILES = [(64, 128, 1024), (100, 77, 650), (1024, 2048, 512), (1100, 1300, 260), (2048, 2176, 256), (2100, 2052, 390),
         (4096, 4096, 640), (2945, 2816, 900), (2050, 8192, 130)]


@pytest.mark.parametrize("m,n,k", TILES)
@pytest.mark.parametrize("b_2d", [True, False])
@pytest.mark.parametrize("out", OUT)
def test_tiles(m, n, k, b_2d, out):
    a, b = F.operand(m, k, False, m + k), F.operand(n, k, b_2d, n)
    F.check_product(nv.fp8_matmul(a, b, out_dtype=out), F.values(a), F.values(b))


def check_groups(counts, align, n, k, out):
    plan = F.plan_of(counts, align)
    a, b = F.operand(plan.rows, k, False, 1), F.operand(n, k, True, 2, lead=(len(counts),))
    d, va, off = nv.fp8_matmul_grouped(a, b, plan, out_dtype=out), F.values(a), H.i64(plan.offsets)
    for e in range(len(counts)):
        F.check_product(d[off[e]:off[e + 1]], va[off[e]:off[e + 1]], F.values(b, e))
    assert not bool(d[off[-1]:].any())


# groups of 1 to 16, 17 to 32, 33 to 64 rows and more, few enough on average for the few-row kernel
@pytest.mark.parametrize("k", [5 * 128, 7 * 128, 11 * 128 - 60, 13 * 128, 23 * 128, 25 * 128])
@pytest.mark.parametrize("out", OUT)
def test_groups_of_few_rows(k, out):
    check_groups([5, 16, 17, 32, 33, 64, 70, 0, 1, 3, 0, 0, 20, 8, 0, 2], 1, 100, k, out)
    check_groups([1, 2, 0, 16, 30, 9, 0, 40], 1, 64, k, out)


# groups whose tiles are 64x64, 64x128, 128x128 and 256x256, and groups that end one row before, at and after a
# half of such a tile
@pytest.mark.parametrize("counts,align,n", [([64, 1, 65, 130], 1, 64), ([63, 128, 129], 16, 200), ([700, 1, 1000], 16, 1000),
                                            ([1500, 127, 1290], 1, 1000), ([1025, 127, 128, 129, 1300, 64], 1, 4096),
                                            ([256, 384, 385, 1, 511, 512, 900], 128, 4096)])
@pytest.mark.parametrize("out", OUT)
def test_groups_in_tiles(counts, align, n, out):
    check_groups(counts, align, n, 300, out)


@pytest.mark.parametrize("m,n", [(64, 64), (500, 500), (700, 1000), (1500, 1536)])
@pytest.mark.parametrize("out", OUT)
def test_weight_gradients(m, n, out):
    plan = F.plan_of([130, 0, 128, 1, 700, 256], 128)
    a, b = F.operand(m, plan.rows, False, 3), F.operand(n, plan.rows, False, 4)
    d, va, vb, off = nv.fp8_matmul_grouped_k(a, b, plan, out_dtype=out), F.values(a), F.values(b), H.i64(plan.offsets)
    for e in range(6):
        F.check_product(d[e], va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]])


# the average that still takes the few-row kernel, and the next one
@pytest.mark.parametrize("counts", [[32] * 8, [40, 24, 32, 31, 33, 31, 64, 1], [33] * 8])
@pytest.mark.parametrize("out", OUT)
def test_groups_around_the_few_row_limit(counts, out):
    check_groups(counts, 1, 200, 1700, out)
