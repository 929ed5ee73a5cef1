"""A mixture-of-experts layer whose products run in block-scaled FP8 or in MXFP4:
forward, backward and the form for a few tokens, from the package's calls alone
(between the two grouped products the activation is torch's).

    python examples/expert_layer.py            # one training step and one decoding step, timed

Each token's row goes to the topk experts that a router chose for it; expert e
computes w2[e] silu(w1[e] x), and the results come back weighted. Weights are
quantized once for each optimizer step, both ways: row-wise for the forward
products, column-wise for the gradients of their inputs. A decoding step of few
tokens takes decode(), one call that reads the same row-wise weights and
quantizes no activation.
"""

from __future__ import annotations

import dataclasses
import os
import sys
from typing import Callable

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_block_scaled_05_amd as nv  # noqa: E402


@dataclasses.dataclass(frozen=True)
class Format:
    """What quantizes, and the products by rows and along k of what it made."""
    quantize: Callable
    grouped: Callable
    grouped_k: Callable


FORMATS = {"fp8": Format(nv.fp8_quantize, nv.fp8_matmul_grouped, nv.fp8_matmul_grouped_k),
           "mxfp4": Format(nv.mxfp4_quantize, nv.mxfp4_matmul_grouped, nv.mxfp4_matmul_grouped_k)}


@dataclasses.dataclass
class Weights:
    """w [experts][n][k], quantized in square blocks in both orientations."""
    row: nv.Fp8Tensor | nv.Mxfp4Tensor
    col: nv.Fp8Tensor | nv.Mxfp4Tensor
    fmt: Format

    @classmethod
    def quantize(cls, w: torch.Tensor, name: str = "fp8") -> "Weights":
        fmt = FORMATS[name]
        return cls(*fmt.quantize(w, columnwise=True, block_2d=True), fmt)


def forward(x, ids, weights, w1: Weights, w2: Weights, *, train: bool):
    """x [tokens][c], ids and weights [tokens][topk] -> [tokens][c], and what
    backward() needs. Without `train` experts' rows are padded to 16, not to the
    128 that the weight gradients need, and nothing is quantized column-wise."""
    f = w1.fmt
    plan = nv.expert_sort(ids, w1.row.data.shape[0], align=128 if train else 16)
    xr, xc = f.quantize(x, columnwise=train, plan=plan)
    h = f.grouped(xr, w1.row, plan)
    ar, ac = f.quantize(torch.nn.functional.silu(h), columnwise=train)
    y = f.grouped(ar, w2.row, plan)
    return nv.expert_combine(y, plan, weights), (plan, xc, h, ac, y)


def backward(dout, weights, w1: Weights, w2: Weights, saved):
    """The gradients of x, the router's weights, w1 and w2 (the last two in FP32)."""
    f, (plan, xc, h, ac, y) = w1.fmt, saved
    dy, dweights = nv.expert_combine_grad(dout, y, plan, weights)
    dyr, dyc = f.quantize(dy, columnwise=True)
    dw2 = f.grouped_k(dyc, ac, plan)
    da = f.grouped(dyr, w2.col, plan)
    s = torch.sigmoid(h.float())
    dh = (da.float() * s * (1 + h.float() * (1 - s))).to(h.dtype)
    dhr, dhc = f.quantize(dh, columnwise=True)
    dw1 = f.grouped_k(dhc, xc, plan)
    dx = nv.expert_gather_grad(f.grouped(dhr, w1.col, plan), plan)
    return dx, dweights, dw1, dw2


def decode(x, ids, weights, w1: Weights, w2: Weights):
    """The forward pass of a few tokens: x as it is, in one call."""
    return nv.expert_mlp(x, ids, weights, w1.row, w2.row, gated=False)


def make(tokens, topk, experts, c, f, seed=0):
    """Seeded inputs: x, ids, weights, w1 [experts][f][c], w2 [experts][c][f]."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    score, ids = torch.randn((tokens, experts), generator=g, device="cuda").topk(topk, dim=1)
    return (randn(tokens, c), ids, torch.softmax(score, 1), randn(experts, f, c, scale=c ** -0.5), randn(experts, c, f, scale=f ** -0.5))


def main() -> None:
    for fmt in FORMATS:
        for name, tokens, kind in (("training step, 8192 tokens", 8192, "train"), ("decoding step, 64 tokens, grouped products", 64, "grouped"),
                                   ("decoding step, 64 tokens, expert_mlp", 64, "decode")):
            x, ids, weights, w1, w2 = make(tokens, 8, 64, 4096, 2048)
            q1, q2 = Weights.quantize(w1, fmt), Weights.quantize(w2, fmt)
            dout = torch.randn_like(x)

            def step():
                if kind == "decode":
                    return decode(x, ids, weights, q1, q2)
                out, saved = forward(x, ids, weights, q1, q2, train=kind == "train")
                return backward(dout, weights, q1, q2, saved) if kind == "train" else out

            for _ in range(3):
                step()
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(10):
                step()
            end.record()
            end.synchronize()
            print(f"{fmt}, {name}, top 8 of 64 experts, 4096 x 2048: {start.elapsed_time(end) / 10:.3f} ms", flush=True)


if __name__ == "__main__":
    main()
