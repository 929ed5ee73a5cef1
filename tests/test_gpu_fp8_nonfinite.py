"""GPU: what infinities and NaN become in block-scaled FP8, byte by byte, and
in a product."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import expert_helpers as H
import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def planted(rows, cols, dtype):
    """Finite values of both signs, zeros among them, and non-finite ones at
    places that blocks of both shapes and orientations meet."""
    x = torch.randn((rows, cols), device=DEV, generator=torch.Generator(DEV).manual_seed(rows + cols))
    x[::5, ::3] = 0
    for r, c, v in ((0, 0, INF), (1, cols - 1, -INF), (2, 1, NAN), (rows - 1, 2, INF), (rows - 1, 5, -INF), (3, 3, INF), (3, 4, NAN),
                    (rows // 2, cols // 2, -INF)):
        x[r, c] = v
    return x.to(dtype)


def check(q, x, block_2d, what):
    with np.errstate(invalid="ignore"):
        want, scales = H.quantize(x, block_2d)
    assert np.array_equal(H.f64(q.scales), scales.astype(np.float64), equal_nan=True), what + " scales"
    assert np.array_equal(H.f64(q.data.to(torch.float32)), want, equal_nan=True), what + " codes"
    codes = q.data.view(torch.uint8).cpu().numpy()
    assert np.array_equal((codes & 0x7F) == 0x7F, np.isnan(want)), what + " bytes"


@pytest.mark.parametrize("rows,cols", [(8, 128), (9, 7), (200, 333), (256, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_2d", [False, True])
def test_codes_of_non_finite_values(rows, cols, dtype, block_2d):
    x = planted(rows, cols, dtype)
    row, col = nv.fp8_quantize(x, columnwise=True, block_2d=block_2d)
    check(row, H.f64(x), block_2d, "row")
    check(col, H.f64(x).T, block_2d, "col")
    # a block with an infinity or a NaN decodes to NaN, whatever its sign
    v = H.values(H.f64(row.data.to(torch.float32)), H.f64(row.scales), block_2d)[:, :cols]
    bad = ~torch.isfinite(row.scales).t().cpu().numpy()
    bad = np.repeat(np.repeat(bad, 128 if block_2d else 1, 0)[:rows], 128, 1)[:, :cols]
    assert np.array_equal(np.isnan(v), bad) and not np.isinf(v).any()


def test_codes_of_non_finite_values_through_a_plan():
    x = planted(40, 200, torch.bfloat16)
    ids = torch.randint(-1, 5, (40, 3), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    plan = nv.expert_sort(ids, 5, align=16)
    row, col = nv.fp8_quantize(x, columnwise=True, plan=plan)
    y = H.f64(nv.expert_gather(x, plan))
    check(row, y, False, "row")
    check(col, y.T, False, "col")


@pytest.mark.parametrize("m,n", [(9, 40), (200, 300)])
def test_product_of_a_row_with_an_infinity_is_nan(m, n):
    g = torch.Generator(DEV).manual_seed(m)
    x, w = torch.randn((m, 256), device=DEV, generator=g), torch.rand((n, 256), device=DEV, generator=g) + 0.5
    x[2, 7], x[5, 200], x[7, 0] = INF, -INF, NAN
    d = nv.fp8_matmul(nv.fp8_quantize(x)[0], nv.fp8_quantize(w, block_2d=True)[0])
    bad = torch.zeros(m, dtype=torch.bool, device=DEV)
    bad[[2, 5, 7]] = True
    assert torch.equal(torch.isnan(d), bad[:, None].expand(m, n)) and not bool(torch.isinf(d).any())
