"""Plain 64-bit forms of the expert-layer operators, in numpy on the host, and
the error bounds that the tests allow.

A rounding to a type is off by at most half a step of the value. Sums in
binary32 of n terms are off by at most n half steps (2^-24) of the sum of
the terms' magnitudes; the matrix core's sum of a block of 128 may also
truncate, which a whole step (2^-23) a term covers."""

from __future__ import annotations

import numpy as np
import torch



def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def i64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.int64).cpu().numpy()


def capacity(slots: int, experts: int, align: int) -> int:
    return (slots + min(experts, slots) * (align - 1)) // align * align


def sort(ids: np.ndarray, experts: int, align: int, rows: int):
    """slot_rows, row_slots, offsets, counts, slot by slot."""
    flat = ids.reshape(-1)
    slot_rows = np.full(flat.size, -1, np.int64)
    row_slots = np.full(rows, -1, np.int64)
    offsets = np.zeros(experts + 1, np.int64)
    counts = np.zeros(experts, np.int64)
    for e in range(experts):
        at = np.nonzero(flat == e)[0]
        counts[e] = at.size
        slot_rows[at] = offsets[e] + np.arange(at.size)
        row_slots[offsets[e]:offsets[e] + at.size] = at
        offsets[e + 1] = offsets[e] + -(-at.size // align) * align
    return slot_rows.reshape(ids.shape), row_slots, offsets, counts


def combine(y: np.ndarray, slot_rows: np.ndarray, w: np.ndarray):
    """The sum, and the sum of the terms' magnitudes."""
    out = np.zeros((slot_rows.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(slot_rows.shape[1]):
        kept = np.nonzero(slot_rows[:, j] >= 0)[0]
        term = w[kept, j:j + 1] * y[slot_rows[kept, j]]
        out[kept] += term
        mag[kept] += np.abs(term)
    return out, mag


def e4m3(v: np.ndarray) -> np.ndarray:
    """The nearest E4M3 value of binary64 v, ties to even, at most 448."""
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def quantize(x: np.ndarray, block_2d: bool):
    """Values and scales of the rows of x [R][C] (binary64 holding binary32
    values): each step of the definition rounded to binary32."""
    r, c = x.shape
    h = 128 if block_2d else 1
    rb, kb = -(-r // h), -(-c // 128)
    v = np.zeros((rb * h, kb * 128), np.float32)
    v[:r, :c] = x.astype(np.float32)
    blocks = v.reshape(rb, h, kb, 128)
    with np.errstate(divide="ignore", over="ignore", under="ignore"):
        s = (np.abs(blocks).max((1, 3)) / np.float32(448)).astype(np.float32)
        e = np.where(s > 0, np.minimum(np.float32(1) / s, np.finfo(np.float32).max), np.float32(0)).astype(np.float32)
        scaled = (blocks * e[:, None, :, None]).astype(np.float32)
    q = e4m3(scaled.astype(np.float64)).reshape(rb * h, kb * 128)[:r]
    return q, np.ascontiguousarray(s.T)


def values(data: np.ndarray, scales: np.ndarray, block_2d: bool) -> np.ndarray:
    """[n][pitch] in binary64."""
    at = np.arange(data.shape[0]) // (128 if block_2d else 1)
    return data * np.repeat(scales.T[at], 128, axis=1)


def product(a: np.ndarray, b: np.ndarray):
    """a b^T in binary64 and the bound of the kernel's binary32 sums: a step a
    term inside a block of 128, half a step a block outside, half a step for
    the product of the scales (twice that, for the sum's rounding as well)."""
    mag = np.abs(a) @ np.abs(b).T
    blocks = max(1, a.shape[1] // 128)
    return a @ b.T, mag * (128 * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24)


def close(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, what: str = "") -> None:
    """got equals want but for `bound` before its last rounding and half a step for that."""
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    half = torch.finfo(got.dtype).eps / 2
    allowed = bound + half * (np.abs(want) + bound) + torch.finfo(got.dtype).tiny
    off = np.abs(g - want)
    assert np.all(off <= allowed), (what, float(np.nanmax(off - allowed)), int(np.sum(~(off <= allowed))))
