"""A mixture-of-experts layer whose products run in block-scaled FP8: forward,
backward and the single-token form, from the package's calls alone (the
activation between the two products is torch's).

    python examples/expert_layer.py            # one training step and one decoding step, timed

Each token's row goes to the topk experts that a router chose for it; expert e
computes w2[e] silu(w1[e] x), and the results come back weighted. Weights are
quantized once for each optimizer step, both ways: row-wise for the forward
products, column-wise for the gradients of their inputs.
"""

from __future__ import annotations

import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_block_scaled_05_amd as nv  # noqa: E402


@dataclasses.dataclass
class Weights:
    """w [experts][n][k], quantized in 128x128 blocks in both orientations."""
    row: nv.Fp8Tensor
    col: nv.Fp8Tensor

    @classmethod
    def quantize(cls, w: torch.Tensor) -> "Weights":
        return cls(*nv.fp8_quantize(w, columnwise=True, block_2d=True))


def forward(x, ids, weights, w1: Weights, w2: Weights, *, train: bool):
    """x [tokens][c], ids and weights [tokens][topk] -> [tokens][c], and what
    backward() needs. Without `train` experts' rows are padded to 16, not to the
    128 that the weight gradients need, and nothing is quantized column-wise."""
    plan = nv.expert_sort(ids, w1.row.data.shape[0], align=128 if train else 16)
    xr, xc = nv.fp8_quantize(x, columnwise=train, plan=plan)
    h = nv.fp8_matmul_grouped(xr, w1.row, plan)
    ar, ac = nv.fp8_quantize(torch.nn.functional.silu(h), columnwise=train)
    y = nv.fp8_matmul_grouped(ar, w2.row, plan)
    return nv.expert_combine(y, plan, weights), (plan, xc, h, ac, y)


def backward(dout, weights, w1: Weights, w2: Weights, saved):
    """The gradients of x, the router's weights, w1 and w2 (the last two in FP32)."""
    plan, xc, h, ac, y = saved
    dy, dweights = nv.expert_combine_grad(dout, y, plan, weights)
    dyr, dyc = nv.fp8_quantize(dy, columnwise=True)
    dw2 = nv.fp8_matmul_grouped_k(dyc, ac, plan)
    da = nv.fp8_matmul_grouped(dyr, w2.col, plan)
    s = torch.sigmoid(h.float())
    dh = (da.float() * s * (1 + h.float() * (1 - s))).to(h.dtype)
    dhr, dhc = nv.fp8_quantize(dh, columnwise=True)
    dw1 = nv.fp8_matmul_grouped_k(dhc, xc, plan)
    dx = nv.expert_gather_grad(nv.fp8_matmul_grouped(dhr, w1.col, plan), plan)
    return dx, dweights, dw1, dw2


def make(tokens, topk, experts, c, f, seed=0):
    """Seeded inputs: x, ids, weights, w1 [experts][f][c], w2 [experts][c][f]."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    score, ids = torch.randn((tokens, experts), generator=g, device="cuda").topk(topk, dim=1)
    return (randn(tokens, c), ids, torch.softmax(score, 1), randn(experts, f, c, scale=c ** -0.5), randn(experts, c, f, scale=f ** -0.5))


def main() -> None:
    for name, tokens, train in (("training step, 8192 tokens", 8192, True), ("decoding step, 64 tokens", 64, False)):
        x, ids, weights, w1, w2 = make(tokens, 8, 64, 4096, 2048)
        q1, q2 = Weights.quantize(w1), Weights.quantize(w2)
        dout = torch.randn_like(x)

        def step():
            out, saved = forward(x, ids, weights, q1, q2, train=train)
            return out if not train else backward(dout, weights, q1, q2, saved)

        for _ in range(3):
            step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            step()
        end.record()
        end.synchronize()
        print(f"{name}, top 8 of 64 experts, 4096 x 2048: {start.elapsed_time(end) / 10:.3f} ms", flush=True)


if __name__ == "__main__":
    main()
