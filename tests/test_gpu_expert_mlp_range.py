"""GPU: the expert layer for a few tokens at the ends of binary32's range, where its results are inside it."""

from __future__ import annotations

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV
from test_gpu_expert_mlp import check, gen, layer

pytestmark = pytest.mark.gpu

# short and long rows, rows of no multiple of eight, few and many slots an expert
SIZES = [(1, 1, 2, 264, 136), (3, 2, 4, 2304, 2200), (5, 2, 4, 333, 129), (40, 2, 2, 1280, 640), (60, 2, 3, 2200, 520), (50, 2, 3, 2051, 260), (100, 3, 64, 256, 1300)]


def given(tokens, topk, experts, cols, seed):
    g = gen(seed)
    x = torch.randn((tokens, cols), device=DEV, generator=g)
    ids = torch.randint(0, experts, (tokens, topk), dtype=torch.int32, device=DEV, generator=g)
    return x, ids, torch.rand((tokens, topk), device=DEV, generator=g)


def run(x, ids, weights, w1, w2, gated, what=""):
    out = nv.expert_mlp(x, ids, weights, w1, w2, gated=gated)
    assert bool(torch.isfinite(out).all()), what
    check(out, x, ids, weights, w1, w2, gated, what)


# ---- FP8 ------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", SIZES)
@pytest.mark.parametrize("gated", [True, False])
def test_fp8_inputs_far_from_one_under_scales_that_make_up_for_them(tokens, topk, experts, cols, hidden, gated):
    # codes times x alone, and their sums over 128 values, leave binary32's range from 100 or so on
    x, ids, weights = given(tokens, topk, experts, cols, 1)
    for far in (95, 110, 118, 124, -100, -118):
        w1, w2 = layer("fp8", experts, cols, hidden, gated, 2)
        w1.scales = (w1.scales.double() * 2.0 ** -far).float()
        run((x * 2.0 ** far).bfloat16(), ids, weights, w1, w2, gated, far)


@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", SIZES)
@pytest.mark.parametrize("gated", [True, False])
def test_fp8_hidden_values_far_from_one(tokens, topk, experts, cols, hidden, gated):
    x, ids, weights = given(tokens, topk, experts, cols, 3)
    for far in (110, 120):
        w1, w2 = layer("fp8", experts, cols, hidden, gated, 4)
        w1.scales *= 2.0 ** (far / 2 if gated else far)
        w2.scales = (w2.scales.double() * 2.0 ** -far).float()
        run(x.bfloat16(), ids, weights, w1, w2, gated, far)


@pytest.mark.parametrize("hidden", [128, 2304])
def test_fp8_every_code_under_every_power_of_two(hidden):
    # each block of 128 rows of the second product's weights has codes 0 .. 126 in turn, for one unit that is not zero and one
    # that is, under a power of two of its own
    codes = torch.arange(127, dtype=torch.uint8, device=DEV)
    powers = torch.arange(-149, 128, device=DEV).double()
    cols, kb = 128 * powers.numel(), hidden // 128
    first = torch.zeros((1, hidden, cols), dtype=torch.uint8, device=DEV)
    first[0, hidden - 5, cols - 3] = 0x38  # 1
    w1 = nv.Fp8Tensor(first.view(torch.float8_e4m3fn), torch.ones((1, cols // 128, kb), device=DEV), hidden, cols, True)
    second = torch.zeros((1, cols, hidden), dtype=torch.uint8, device=DEV)
    for unit in (hidden - 5, hidden - 4):
        second[0].view(-1, 128, hidden)[:, :127, unit] = codes
    w2 = nv.Fp8Tensor(second.view(torch.float8_e4m3fn), torch.exp2(powers).float().expand(1, kb, -1).contiguous(), cols, hidden, True)
    value = codes.view(torch.float8_e4m3fn).double()
    ids, weights = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV)
    for power in (30, 60):
        x = torch.zeros((1, cols), dtype=torch.bfloat16, device=DEV)
        x[0, cols - 3] = 2.0 ** power  # silu leaves it as it is
        out = nv.expert_mlp(x, ids, weights, w1, w2, gated=False).reshape(-1, 128)
        want = (torch.exp2(powers)[:, None] * value * 2.0 ** power).float().bfloat16()
        assert torch.equal(out[:, :127], want), power
        assert not bool(out[:, 127].any())
