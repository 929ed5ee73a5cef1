"""GPU: the expert layer for a few tokens at the ends of binary32's range, where its results are inside it."""

from __future__ import annotations

import pytest
import torch

import mxfp4_helpers as M
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


# ---- MXFP4 ----------------------------------------------------------------------

CODES = torch.tensor(list(M.E2M1) + list(-M.E2M1), dtype=torch.float64)
SCALES = (0, 1, 2, 127, 251, 252, 253, 254)


def table(rows_at, pitch, n):
    """Rows of every code under every scale of SCALES, at value 32 q of a row for q = row % 4 (of block `rows_at`), and again at the
    value after it: an Mxfp4Tensor of n rows, and each row's value and q."""
    kb = pitch // 128
    data = torch.zeros((1, n, pitch // 2), dtype=torch.uint8)
    scales = torch.full((1, kb, n, 4), 127, dtype=torch.uint8)
    value, place = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.long)
    for r in range(n):
        code, s, q = r // 4 % 16, SCALES[r // 64 % len(SCALES)], r % 4
        at = 128 * rows_at + 32 * q
        data[0, r, at // 2] = code | code << 4
        scales[0, rows_at, r, q] = s
        value[r], place[r] = CODES[code] * 2.0 ** (s - 127), at
    return data, scales, value.to(DEV), place.to(DEV)


ROWS = 4 * 16 * len(SCALES)


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("cols", [512, 2304, 4224])
@pytest.mark.parametrize("gated", [True, False])
def test_every_code_under_the_scales_of_both_ends_in_the_first_product(tokens, cols, gated):
    data, scales, value, place = table(1, cols, ROWS)
    if gated:  # the second half's rows are 1 in the first column
        up, ups = torch.zeros_like(data), torch.full_like(scales, 127)
        up[0, :, 0] = 2
        data, scales = torch.cat([data, up], 1), torch.cat([scales, ups], 2)
    w1 = nv.Mxfp4Tensor(data.to(DEV), scales.to(DEV), (1 + gated) * ROWS, cols)
    w2 = nv.mxfp4_quantize(torch.eye(cols, ROWS, device=DEV)[None])[0]
    ids, weights = torch.zeros((tokens, 1), dtype=torch.int32, device=DEV), torch.ones((tokens, 1), device=DEV)
    for power in (-100, -4):
        x = torch.zeros((tokens, cols), dtype=torch.bfloat16, device=DEV)
        x[:, 0], x[:, 128:256:32] = 1, 2.0 ** power  # (the value next to each is zero)
        out = nv.expert_mlp(x, ids, weights, w1, w2, gated=gated)[:, :ROWS].double()
        v = value * 2.0 ** power  # (at most 6 * 2^123)
        want = v * torch.sigmoid(v)
        # an exponential is off by a few 2^-24 for each unit of its argument, of which 100 count
        miss = (out - want).abs()
        assert bool((miss <= want.abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -126).all()), power


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("hidden", [256, 2304])
def test_every_code_under_the_scales_of_both_ends_in_the_second_product(tokens, hidden):
    data, scales, value, place = table(1, hidden, ROWS)
    w1 = torch.zeros((1, hidden, ROWS), device=DEV)
    w1[0, 128:256:32, 5] = 1
    w1, w2 = nv.mxfp4_quantize(w1)[0], nv.Mxfp4Tensor(data.to(DEV), scales.to(DEV), ROWS, hidden)
    ids, weights = torch.zeros((tokens, 1), dtype=torch.int32, device=DEV), torch.ones((tokens, 1), device=DEV)
    for power, h in ((-40, -41), (40, 40)):  # silu halves what is small and leaves what is large
        x = torch.zeros((tokens, ROWS), dtype=torch.bfloat16, device=DEV)
        x[:, 5] = 2.0 ** power
        out = nv.expert_mlp(x, ids, weights, w1, w2, gated=False)
        want = (value * 2.0 ** h).float().bfloat16()
        assert torch.equal(out, want.expand(tokens, -1)), power


@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", SIZES)
@pytest.mark.parametrize("gated", [True, False])
def test_mxfp4_weights_of_the_largest_scales(tokens, topk, experts, cols, hidden, gated):
    x, ids, weights = given(tokens, topk, experts, cols, 5)
    x[:, ::3] = 0
    for first in (True, False):
        w1, w2 = layer("mxfp4", experts, cols, hidden, gated, 6)
        q = w1 if first else w2
        q.scales = torch.randint(249, 255, q.scales.shape, device=DEV, generator=gen(7)).to(torch.uint8)
        # x or h makes up for them: the products' sums, and h of a gated layer, stay inside
        run((x * 2.0 ** (-110 if first else -50 if gated else -100)).bfloat16(), ids, weights, w1, w2, gated, first)


@pytest.mark.parametrize("tokens", [1, 50])
@pytest.mark.parametrize("cols", [200, 2300])
def test_mxfp4_rows_under_nan(tokens, cols):
    x, ids, weights = given(tokens, 1, 3, cols, 8)
    w1, w2 = layer("mxfp4", 3, cols, 264, True, 9)
    want = nv.expert_mlp(x.bfloat16(), ids, weights, w1, w2)
    w2.scales[1, 1, 77, 3] = 255
    out = nv.expert_mlp(x.bfloat16(), ids, weights, w1, w2)
    nan = torch.zeros((tokens, cols), dtype=torch.bool, device=DEV)
    nan[:, 77] = ids[:, 0] == 1
    assert torch.equal(torch.isnan(out), nan) and torch.equal(out[~nan], want[~nan])
    w1.scales[2, 0, 264 + 100, 0] = 255  # one unit, which every column takes
    out = nv.expert_mlp(x.bfloat16(), ids, weights, w1, w2)
    nan[ids[:, 0] == 2] = True
    assert torch.equal(torch.isnan(out), nan) and torch.equal(out[~nan], want[~nan])


# ---- both -----------------------------------------------------------------------

def one_layer(kind, gate, up, out):
    """Weights for 128 columns and 32 units, of one expert: unit 0's gate (and its up row, if any) as {column: power of two}, and row c of
    w2 the power of two out[c] for unit 0; row c of w2 that is not in out is zero."""
    units = 32 if up is None else 64

    def pack(rows, n, k):
        if kind == "fp8":
            kb = 1
            data = torch.zeros((1, n, 128), dtype=torch.uint8, device=DEV)
            powers = {p for at in rows.values() for p in at.values()}
            assert len(powers) == 1  # one block's scale
            for r, at in rows.items():
                for c in at:
                    data[0, r, c] = 0x38
            return nv.Fp8Tensor(data.view(torch.float8_e4m3fn), torch.full((1, kb, 1), 2.0 ** powers.pop(), device=DEV), n, k, True)
        data = torch.zeros((1, n, 64), dtype=torch.uint8, device=DEV)
        scales = torch.full((1, 1, n, 4), 127, dtype=torch.uint8, device=DEV)
        for r, at in rows.items():
            for c, p in at.items():
                data[0, r, c // 2] |= 2 << (4 * (c % 2))
                scales[0, 0, r, c // 32] = 127 + p
        return nv.Mxfp4Tensor(data, scales, n, k)

    rows = {0: gate} if up is None else {0: gate, 32: up}
    return pack(rows, units, 128), pack({c: {0: p} for c, p in out.items()}, 128, 32)


@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
def test_hidden_values_next_to_the_largest_number(kind):
    # h between the largest BF16 number and the largest of binary32
    most = 255 * 2.0 ** 120
    w1, w2 = one_layer(kind, {0: 0, 1: 0}, None, {3: -20, 7: -20})
    more = [0.0, 0.25, 0.5, 0.75, 0.96875]
    x = torch.zeros((len(more), 128), dtype=torch.float64)
    x[:, 0], x[:, 1] = most, torch.tensor(more) * 2.0 ** 120
    ids, weights = torch.zeros((len(more), 1), dtype=torch.int32, device=DEV), torch.ones((len(more), 1), device=DEV)
    out = nv.expert_mlp(x.bfloat16().to(DEV), ids, weights, w1, w2, gated=False)
    want = (x.sum(1) * 2.0 ** -20).float().bfloat16().to(DEV)
    keep = torch.zeros(128, dtype=torch.bool, device=DEV)
    keep[3] = keep[7] = True
    assert torch.equal(out[:, keep], want[:, None].expand(-1, 2))
    assert not bool(out[:, ~keep].any())


@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
def test_gates_far_below_zero(kind):
    # silu(g) = g e^g is small there, not nothing: times u of 2^100 it is a number to be seen
    gates = torch.tensor([-60.0, -79, -80, -80.5, -81, -87, -88, -88.5, -89, -90, -91, -95, -100, -103, -110, -200, -1000], dtype=torch.float64)
    w1, w2 = one_layer(kind, {0: 0}, {1: 0}, {3: 0})
    x = torch.zeros((gates.numel(), 128), dtype=torch.float64)
    x[:, 0], x[:, 1] = gates, 2.0 ** 100
    assert torch.equal(x.bfloat16().double(), x)
    ids, weights = torch.zeros((gates.numel(), 1), dtype=torch.int32, device=DEV), torch.ones((gates.numel(), 1), device=DEV)
    out = nv.expert_mlp(x.bfloat16().to(DEV), ids, weights, w1, w2)[:, 3].double().cpu()
    want = gates * torch.exp(gates) * 2.0 ** 100  # (1 + e^g is 1)
    # an exponential is off by a few 2^-24 for each unit of its argument; silu is a binary32 number, of steps of 2^-149 at least
    assert bool(((out - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** (100 - 148)).all()), (out, want)
