"""Plain 64-bit forms of MXFP4 quantization and products, and the error bound
that the product tests allow.

An instruction of the matrix cores sums 64 or 128 products of codes, times powers
of two, into an accumulator. Aligning the blocks' sums and rounding the result to
binary32 puts it off by at most a step (2^-23) of the magnitudes that it sums."""

from __future__ import annotations

import numpy as np
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1(v: np.ndarray) -> np.ndarray:
    """The nearest E2M1 value of binary64 v, middles to the even code, at most 6; of zeros and of what becomes 0 the sign stays."""
    m = np.abs(v)
    code = np.zeros(v.shape, np.int64)
    for i in range(7):
        middle = (E2M1[i] + E2M1[i + 1]) / 2
        code += (m > middle) | ((m == middle) & (i % 2 == 1))
    return np.copysign(E2M1[code], v)


def quantize(x: np.ndarray, block_2d: bool):
    """Values over their scale [R][pitch] and scale bytes [ceil(C / 128)][R][4] of the rows of x [R][C] (binary64)."""
    r, c = x.shape
    h = 32 if block_2d else 1
    rb, pitch = -(-r // h), -(-c // 128) * 128
    v = np.zeros((rb * h, pitch))
    v[:r, :c] = x
    blocks = v.reshape(rb, h, pitch // 32, 32)
    m = np.abs(blocks).max((1, 3))
    finite = np.isfinite(m)  # an infinity or a NaN in the block: not so
    _, e = np.frexp(np.where(finite, m, 1.0))  # m in 2^(e - 1) .. 2^e
    s = np.where(m > 0, np.maximum(e - 1 + 127 - 2, 0), 0)
    s = np.where(finite, s, 255)
    scale = np.exp2(np.where(finite, s, 127) - 127.0)
    q = e2m1(np.where(finite[:, None, :, None], blocks, 0.0) / scale[:, None, :, None]).reshape(rb * h, pitch)[:r]
    s = np.repeat(s, h, 0)[:r].reshape(r, pitch // 128, 4)
    return q, np.ascontiguousarray(s.transpose(1, 0, 2))


def codes(data: torch.Tensor) -> np.ndarray:
    """The values over their scale, with the sign of zeros, of bytes [..][pitch / 2]."""
    d = data.cpu().numpy()
    code = np.stack([d & 15, d >> 4], -1).reshape(*d.shape[:-1], -1)
    return np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]


def values(q: nv.Mxfp4Tensor, b=None) -> torch.Tensor:
    """The values [n][pitch] in binary64, on the device (of matrix b of a batch)."""
    data, scales = (q.data, q.scales) if b is None else (q.data[b], q.scales[b])
    table = torch.tensor(np.concatenate([E2M1, -E2M1]), device=data.device)
    v = table[torch.stack([data & 15, data >> 4], -1).reshape(data.shape[0], 2 * data.shape[1]).long()]
    s = scales.transpose(0, 1).reshape(data.shape[0], 4 * scales.shape[0]).double()
    s = torch.where(s == 255, torch.nan, torch.exp2(s - 127))
    return v * s.repeat_interleave(32, 1)


def operand(n, k, seed, lead=(), exponents=(0, 0), block_2d=False):
    """Quantized normal rows with a factor per column; each block's scale times a power of two of its own, with an
    exponent from `exponents`, first and last."""
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn((*lead, n, k), device=DEV, generator=g) * torch.exp(torch.randn(k, device=DEV, generator=g))
    q = nv.mxfp4_quantize(x, block_2d=block_2d)[0]
    if exponents != (0, 0):
        up = torch.randint(exponents[0], exponents[1] + 1, q.scales.shape, device=DEV, generator=g)
        q.scales = (q.scales.int() + up).clamp(0, 254).to(torch.uint8)
    return q


def check_product(d: torch.Tensor, a: torch.Tensor, b: torch.Tensor, what="") -> None:
    """d against a b^T for a [m][k] and b [n][k] in binary64, of magnitudes that binary32 holds: an instruction each
    64 values at most, and up to eight sums of shares that are added up."""
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    assert d.shape == want.shape, what
    f = torch.finfo(d.dtype)
    bound = mag * 2.0 ** -23 * (-(-a.shape[1] // 64) + 8)
    allowed = bound + f.eps / 2 * (want.abs() + bound) + f.smallest_normal * f.eps + 2.0 ** -148
    off = (d.double() - want).abs()
    assert bool((off <= allowed).all()), (what, int((~(off <= allowed)).sum()), float((off - allowed).max()))
    assert bool((d[mag == 0] == 0).all()), what
