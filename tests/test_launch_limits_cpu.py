"""Products whose launch would need 2^32 threads or more are refused as a shape,
before anything reaches a GPU."""

from __future__ import annotations

import pytest

import nvfp4_block_scaled_05_amd as nv

P = 0x100000  # a fake, aligned device address


@pytest.mark.parametrize("m,n,k", [
    ((1 << 31) - 1, 1, 1),    # 2^24 tiles of 128 rows, 256 threads each
    ((1 << 31) - 1, 1, 0),    # the same where only zeros are written
    (1, (1 << 31) - 1, 1),    # few rows: 2^26 tiles of 32 columns, one wave each
    (32, 1 << 28, 26 * 128),  # few rows, eight waves each
])
@pytest.mark.parametrize("b_2d", [0, 1])
def test_dense(m, n, k, b_2d):
    q = nv.nvfp4_fp8_t(P, P)
    assert nv.load().nvfp4_fp8_matmul(q, q, m, n, k, b_2d, P, nv.NVFP4_IN_BF16, None) == nv.NVFP4_ERR_SHAPE
    assert "too large for one launch" in nv.nvfp4_last_error()


def test_grouped():
    q = nv.nvfp4_fp8_t(P, P)
    lib = nv.load()
    assert lib.nvfp4_fp8_matmul_grouped(q, q, P, 4, (1 << 31) - 1, 1, 128, P, nv.NVFP4_IN_BF16, None) == nv.NVFP4_ERR_SHAPE
    assert lib.nvfp4_fp8_matmul_grouped_k(q, q, P, 256, 1 << 23, 1, 128, P, nv.NVFP4_IN_FP32, None) == nv.NVFP4_ERR_SHAPE
    assert "too large for one launch" in nv.nvfp4_last_error()
