"""GPU: calls whose launches need 2^32 threads and more."""

from __future__ import annotations

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def test_rows_of_more_tokens_than_one_grid_line_has_waves():
    # whole numbers small enough for every step to be exact
    tokens, cols = (1 << 26) + 5, 4
    g = torch.Generator(DEV).manual_seed(1)
    ids = torch.randint(-1, 2, (tokens, 1), dtype=torch.int32, device=DEV, generator=g)
    x = torch.randint(-4, 5, (tokens, cols), device=DEV, generator=g, dtype=torch.int8).to(torch.bfloat16)
    w = torch.full((tokens, 1), 2.0, device=DEV)
    plan = nv.expert_sort(ids, 2, align=16)
    at = plan.slot_rows[:, 0].long()
    kept = at >= 0
    y = nv.expert_gather(x, plan)
    assert torch.equal(y[at[kept]], x[kept]) and not bool(y[plan.row_slots < 0].any())
    out = nv.expert_combine(y, plan, w)
    assert torch.equal(out, torch.where(kept[:, None], 2 * x, 0))
    dy, dw = nv.expert_combine_grad(x, y, plan, w)
    assert torch.equal(dy[at[kept]], 2 * x[kept]) and not bool(dy[plan.row_slots < 0].any())
    assert torch.equal(dw[:, 0], torch.where(kept, x.float().square().sum(1), 0))


@pytest.mark.parametrize("block_2d", [False, True])
def test_quantize_of_more_matrices_than_one_grid_line_has_tiles(block_2d):
    batch = (1 << 24) + 3
    x = torch.randn((batch, 1, 1), device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(torch.bfloat16)
    row, col = nv.fp8_quantize(x, columnwise=True, block_2d=block_2d)
    for q in (row, col):
        assert torch.equal(q.scales[:, 0, 0], x[:, 0, 0].float().abs() / torch.full((), 448.0, device=DEV))
        codes = q.data.view(torch.uint8)[:, 0]
        code = torch.where(x[:, 0, 0] == 0, 0, 0x7E).to(torch.uint8) | (x[:, 0, 0].view(torch.int16) < 0).to(torch.uint8) * 128
        assert torch.equal(codes[:, 0], code)
        assert not bool(codes[:, 1:].any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_scaled_tensor_of_more_rows_than_one_grid_line_has(dtype):
    rows, cols, tail = (1 << 24) + 256, 16, 512
    x = torch.randn((rows, cols), device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(dtype)
    amax = x.float().abs().amax(1)
    row, _ = nv.quantize(x, columnwise=False, cfg=nv.make_config(row_scaled=True))
    assert torch.equal(row.amax, amax)
    last, _ = nv.quantize(x[-tail:].contiguous(), columnwise=False, cfg=nv.make_config(row_scaled=True))
    assert torch.equal(row.data[-tail:], last.data) and torch.equal(row.scales[-tail:], last.scales)
    only = torch.zeros(rows, device=DEV)
    nv.nvfp4_compute_amax(x, only, None, nv.make_config(row_scaled=True))
    assert torch.equal(only, amax)


def test_row_scaled_groups_of_more_rows_than_one_grid_line_has():
    rows, cols, tail = (1 << 24) + 256, 16, 512
    x = torch.randn((rows, cols), device=DEV, generator=torch.Generator(DEV).manual_seed(4)).to(torch.bfloat16)
    cfg = dict(row_scaled=True, stochastic=True, sr_seed=3)
    row, _ = nv.quantize_grouped(x, [rows - tail, tail], columnwise=False, cfg=nv.make_config(**cfg))
    assert torch.equal(row.amax, x.float().abs().amax(1))
    last, _ = nv.quantize_grouped(x[-tail:].contiguous(), [tail], columnwise=False, cfg=nv.make_config(**cfg))
    assert torch.equal(row.data[-tail * cols // 2:], last.data) and torch.equal(row.scales[-tail * cols // 16:], last.scales)
