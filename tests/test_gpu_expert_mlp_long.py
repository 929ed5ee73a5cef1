"""GPU: the expert layer for a few tokens with rows of many segments and more slots an expert than a pass takes."""

from __future__ import annotations

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV
from test_gpu_expert_mlp import check, gen, layer

pytestmark = pytest.mark.gpu

SIZES = [(40, 1, 2, 256, 8192), (36, 2, 3, 264, 12296), (70, 1, 2, 128, 16384), (34, 2, 2, 12288, 200), (50, 1, 2, 16392, 136), (40, 2, 2, 8201, 130),
         (45, 1, 1, 8192, 8200), (256, 2, 2, 4104, 2056)]


@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", SIZES)
@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [True, False])
def test_long_rows_and_many_slots(tokens, topk, experts, cols, hidden, kind, gated):
    g = gen(tokens + cols)
    x = torch.randn((tokens, cols), device=DEV, generator=g).bfloat16()
    ids = torch.randint(0, experts, (tokens, topk), dtype=torch.int32, device=DEV, generator=g)
    ids[tokens // 3, 0] = -1
    weights = torch.rand((tokens, topk), device=DEV, generator=g)
    w1, w2 = layer(kind, experts, cols, hidden, gated, hidden)
    out = nv.expert_mlp(x, ids, weights, w1, w2, gated=gated)
    check(out, x, ids, weights, w1, w2, gated)
    assert torch.equal(nv.expert_mlp(x, ids, weights, w1, w2, gated=gated), out)
