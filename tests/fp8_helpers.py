"""Block-scaled FP8 operands, plans and 64-bit products on the device, for
sizes whose comparison on the host would take long. The bounds are
expert_helpers.product's and expert_helpers.close's."""

from __future__ import annotations

import numpy as np
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV


def operand(n, k, block_2d, seed, lead=(), exponents=(0, 0)):
    """Quantized normal rows with a factor per column; each block's scale times a power of two of its own, with
    an exponent from `exponents`, first and last."""
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn((*lead, n, k), device=DEV, generator=g) * torch.exp(torch.randn(k, device=DEV, generator=g))
    q = nv.fp8_quantize(x, block_2d=block_2d)[0]
    q.scales *= torch.exp2(torch.randint(exponents[0], exponents[1] + 1, q.scales.shape, device=DEV, generator=g).float())
    return q


def values(q, b=None):
    """The values [n][pitch] in binary64 (of matrix b of a batch)."""
    data, scales = (q.data, q.scales) if b is None else (q.data[b], q.scales[b])
    s = scales.double().t().repeat_interleave(128, 1)
    if q.block_2d:
        s = s.repeat_interleave(128, 0)[:data.shape[0]]
    return data.float().double() * s


def plan_of(counts, align, seed=0):
    """A plan whose experts get these many slots."""
    ids = np.concatenate([np.full(c, e, np.int32) for e, c in enumerate(counts)])
    np.random.default_rng(seed).shuffle(ids)
    return nv.expert_sort(torch.from_numpy(ids.reshape(-1, 1)).to(DEV), len(counts), align=align)


def check_product(d, a, b):
    """d against a b^T for a [m][k] and b [n][k] in binary64, wherever no sum of FP32 on the way can overflow;
    an infinity of its sign where blocks of one sign alone, each as far off as its sum can be, are past the
    largest FP32 number."""
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    bound = mag * (128 * 2.0 ** -23 + (max(1, a.shape[1] // 128) + 2) * 2.0 ** -24)
    f = torch.finfo(d.dtype)
    steps = a.shape[1] // 128 * 2.0 ** -149 + f.smallest_normal * f.eps  # of subnormal numbers: a block's term, and the result
    allowed = bound + f.eps / 2 * (want.abs() + bound) + steps
    fits = mag < 2.0 ** 126
    ok = (d.double() - want).abs() <= allowed
    assert bool((ok | ~fits).all()), (int((~ok & fits).sum()), float(((d.double() - want).abs() - allowed)[fits & ~ok].max()))
    assert bool((d[mag == 0] == 0).all())
    if bool(fits.all()):
        return
    up, down = torch.zeros_like(want), torch.zeros_like(want)
    for at in range(0, a.shape[1], 128):
        term = a[:, at:at + 128] @ b[:, at:at + 128].t()
        up += term.clamp(min=0)
        down += (-term).clamp(min=0)
    assert bool((d[(up - bound > 2.0 ** 129) & (down + bound < 2.0 ** 126)] == float("inf")).all())
    assert bool((d[(down - bound > 2.0 ** 129) & (up + bound < 2.0 ** 126)] == -float("inf")).all())
