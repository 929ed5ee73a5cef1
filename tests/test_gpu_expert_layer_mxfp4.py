"""GPU: the example expert layer in MXFP4 against the same layer in 64 bits:
a training step, its gradients, the updated weights, and decoding with them."""

from __future__ import annotations

import os
import sys

import pytest
import torch

import mxfp4_helpers as M
import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV
from test_gpu_expert_layer import exact, rel

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as layer  # noqa: E402

pytestmark = pytest.mark.gpu

# What quantization to E2M1 is off by, for normal values whose block has its largest one at t (4 <= t < 8): a code's half
# step is 0.25 below 2, 0.5 below 4, 1 up to 6, and what is above 6 becomes 6. A block of 32 has its largest at 2.1 deviations
# or so, 32x32 at 3.2, so a deviation is 1.25 (t = 4, 1024 values) to 3.8 (t = 8, 32 values). Errors are spread evenly over a
# step. Deviation 1.25: 0.25 / sqrt(3) = 0.144 with nine tenths of the values, 0.29 with the rest: 0.16 / 1.25 = 0.13 of it.
# Deviation 3.8: parts 0.40, 0.31, 0.18 and 0.11 of the values, mean squares 0.021, 0.083, 0.33 and 4 / 3: 0.49 / 3.8 = 0.13.
# A product of two such operands: 0.18; no result passes through more than three.
OFF = 3 * 0.18


def step(tokens, topk, experts, c, f, dropped=False):
    x, ids, weights, w1, w2 = layer.make(tokens, topk, experts, c, f, seed=tokens)
    if dropped:
        ids[::5, 0] = -1
        ids[3] = -1
    q1, q2 = layer.Weights.quantize(w1, "mxfp4"), layer.Weights.quantize(w2, "mxfp4")
    out, saved = layer.forward(x, ids, weights, q1, q2, train=True)
    dout = torch.randn(out.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(out.dtype)
    return (x, ids, weights, w1, w2), (q1, q2), out, saved, dout, layer.backward(dout, weights, q1, q2, saved)


@pytest.mark.parametrize("tokens,topk,experts,c,f", [(300, 3, 5, 256, 384), (70, 2, 16, 200, 136), (33, 4, 4, 520, 96)])
@pytest.mark.parametrize("dropped", [False, True])
def test_training_step(tokens, topk, experts, c, f, dropped):
    given, _, out, _, dout, grads = step(tokens, topk, experts, c, f, dropped)
    x, ids, weights, w1, w2 = given
    want, leaves = exact(*given)
    want.backward(dout.double())
    assert rel(out, want.detach()) < OFF
    for got, leaf, name in zip(grads, leaves, ("x", "weights", "w1", "w2")):
        assert got.shape == leaf.shape and rel(got, leaf.grad) < OFF, name
    # against differences of the 64-bit layer along each gradient: <exact, got> is within OFF |exact| |got| of |got|^2
    for i, got in enumerate(grads):
        place = (0, 2, 3, 4)[i]
        d = got.double() / got.double().norm()
        eps = 1e-4

        def loss(sign):
            moved = [t.double() if t.is_floating_point() else t for t in given]
            moved[place] = moved[place] + sign * eps * d
            return float((exact(*moved)[0].detach() * dout.double()).sum())

        slope, norm = (loss(1) - loss(-1)) / (2 * eps), float(got.double().norm())
        assert abs(slope - norm) <= OFF * float(leaves[i].grad.norm()) * 1.01


def test_weight_gradients_are_the_products_of_what_was_quantized():
    given, (_, q2), _, (plan, xc, h, ac, y), dout, (_, _, dw1, dw2) = step(200, 2, 6, 264, 160)
    dy, _ = nv.expert_combine_grad(dout, y, plan, given[2])
    dyr, dyc = nv.mxfp4_quantize(dy, columnwise=True)
    off = plan.offsets.tolist()
    for e in range(6):
        rows = slice(off[e], off[e + 1])
        M.check_product(dw2[e], M.values(dyc)[:, rows], M.values(ac)[:, rows], f"dw2 {e}")
        if off[e] == off[e + 1]:
            continue
        s = torch.sigmoid(h[rows].double())
        dh = (M.values(dyr)[rows] @ M.values(q2.col, e).t()) * s * (1 + h[rows].double() * (1 - s))
        # (dh is quantized before its product: what one operand is off by, and BF16's roundings)
        assert rel(dw1[e], dh.t() @ M.values(xc)[:, rows].t()) < OFF / 3, e


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("tokens", [1, 16, 120])
def test_update_and_decode(fmt, tokens):
    """A step of the optimizer, the weights quantized again, and tokens decoded with them, as one captured run too."""
    x, ids, weights, w1, w2 = layer.make(256, 2, 8, 512, 256, seed=2)
    q1, q2 = layer.Weights.quantize(w1, fmt), layer.Weights.quantize(w2, fmt)
    out, saved = layer.forward(x, ids, weights, q1, q2, train=True)
    _, _, dw1, dw2 = layer.backward(out, weights, q1, q2, saved)
    w1, w2 = (w1 - 1e-3 * dw1).bfloat16(), (w2 - 1e-3 * dw2).bfloat16()
    x, ids, weights, _, _ = layer.make(tokens, 2, 8, 512, 256, seed=3)

    def run():
        p1, p2 = layer.Weights.quantize(w1, fmt), layer.Weights.quantize(w2, fmt)
        return layer.decode(x, ids, weights, p1, p2), layer.forward(x, ids, weights, p1, p2, train=False)[0]

    one, grouped = run()
    want = exact(x, ids, weights, w1, w2)[0].detach()
    # the weights' rounding alone, twice; the activations' as well
    assert rel(one, want) < 2 * (0.13 if fmt == "mxfp4" else 0.036) + 0.004
    assert rel(grouped, want) < (OFF if fmt == "mxfp4" else 3 * 0.051)
    assert rel(one, want) < rel(grouped, want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        static = run()
    g = torch.Generator(DEV).manual_seed(4)
    for i in range(3):
        x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        w1.copy_(w1 * 1.01)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(static, run())), i
