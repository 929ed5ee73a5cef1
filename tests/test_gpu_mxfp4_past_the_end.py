"""GPU: rows past the last group's, in memory that held something else, for every kernel that products by groups of rows choose."""

from __future__ import annotations

import pytest
import torch

import mxfp4_helpers as M
import nvfp4_block_scaled_05_amd as nv
from fp8_helpers import plan_of
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

# 64x128 tiles, 128x128, 256x256
CASES = [([5, 0, 20], 16, 190, 96, 300), ([100, 0, 129], 128, 1000, 520, 260), ([1100, 0, 300], 128, 5000, 4100, 130), ([0, 0, 0], 16, 130, 136, 128)]


@pytest.mark.parametrize("counts,align,rows,n,k", CASES)
@pytest.mark.parametrize("out,code", [(torch.bfloat16, nv.NVFP4_IN_BF16), (torch.float32, nv.NVFP4_IN_FP32)])
@pytest.mark.parametrize("fill", [0x5A, 0xFF])
def test_rows_past_the_last_group_are_cleared(counts, align, rows, n, k, out, code, fill):
    few = plan_of(counts, align)
    ids = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32, device=DEV), torch.tensor(counts, device=DEV))[:, None]
    plan = nv.expert_sort(ids, len(counts), align=align, rows=rows)
    assert torch.equal(plan.offsets, few.offsets)
    end = plan.offsets.tolist()[-1]
    a, b = M.operand(rows, k, 1), M.operand(n, k, 2, lead=(len(counts),))
    a.scales[:, end:] = 255  # what those rows hold of a does not count
    size = rows * n * torch.finfo(out).bits // 8
    whole = torch.full((size + 512,), fill, dtype=torch.uint8, device=DEV)
    part = whole[256:256 + size]
    assert nv.load().nvfp4_mxfp4_matmul_grouped(a.as_c(), b.as_c(), plan.offsets.data_ptr(), len(counts), rows, n, k, part.data_ptr(), code,
                                                torch.cuda.current_stream().cuda_stream) == nv.NVFP4_OK
    d = part.view(out).reshape(rows, n)
    assert not bool(part.reshape(rows, -1)[end:].any())
    assert bool((whole[:256] == fill).all()) and bool((whole[256 + size:] == fill).all())
    off, va = plan.offsets.tolist(), M.values(a)
    for e in range(len(counts)):
        if off[e] < off[e + 1]:
            M.check_product(d[off[e]:off[e + 1]], va[off[e]:off[e + 1]], M.values(b, e), f"group {e}")
