"""Rotary positions, cache rows and attention in float64, written from the
formulas of include/wal.h (numpy only, nothing shared with the library).

Every function that stands for a kernel with fp32 sums or bf16 operands also
gives what its error bound is made of, so that a test states its tolerance
per element instead of choosing one.
"""
from __future__ import annotations

import numpy as np


def rope_freqs(rot, base, scaling="plain", factor=1.0, trained_len=0.0, turns_low=1.0, turns_high=32.0):
    """Radians per position of each pair, and the magnitude."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        g = np.clip((trained_len * f / (2 * np.pi) - turns_low) / (turns_high - turns_low), 0.0, 1.0)
        return f * g + f / factor * (1.0 - g), 0.1 * np.log(factor) + 1.0
    return f, 1.0


def rope(x, pos, freqs, magnitude=1.0, interleaved=False):
    """x [n][heads][dim] -> (rotated, |a| + |b| of each rotated element's pair times the magnitude; 0 where copied)."""
    x = np.asarray(x, np.float64)
    r = 2 * len(freqs)
    a = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    b = a + 1 if interleaved else a + r // 2
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(freqs, np.float64)[None]
    c, s = (magnitude * np.cos(ang))[:, None], (magnitude * np.sin(ang))[:, None]
    out, size = x.copy(), np.zeros_like(x)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = magnitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, size


def int8_rows(x):
    """Rows (last axis) as int8 codes and fp32 scales, in the fp32 arithmetic that include/wal.h states."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        ok = np.isfinite(x).all(-1)
        live = ok & (top >= np.float32(2.0 ** -100))
        scale = np.where(live, top * np.float32(1.0 / 127.0), np.float32(0.0))
        inv = np.where(live, np.float32(127.0) / top, np.float32(0.0))
        codes = np.where(live[..., None], np.rint(x * inv[..., None]), 0.0).astype(np.int8)
    return codes, np.where(ok, scale, np.float32(np.nan)).astype(np.float32)


def attend(q, k, v, last, scale, present=None):
    """q [rows][heads][dim] over k, v [keys][kv heads][dim]: row i sees the keys
    j <= last[i] (of those present).  Returns the output, the sums of w_j |v_j|
    and, per row and head, the largest sum of |scale q_e k_je| over seen keys."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    group = q.shape[1] // k.shape[1]
    seen = np.arange(k.shape[0])[None] <= np.asarray(last)[:, None]
    if present is not None:
        seen = seen & np.asarray(present, bool)[None]
    out, size, most = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
    for h in range(q.shape[1]):
        kh, vh = k[:, h // group], v[:, h // group]
        x = np.where(seen, scale * (q[:, h] @ kh.T), -np.inf)
        top = x.max(-1, initial=-np.inf, keepdims=True)
        w = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
        total = w.sum(-1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
        out[:, h], size[:, h] = w @ vh, w @ np.abs(vh)
        if k.shape[0]:
            most[:, h] = np.where(seen, abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T), 0.0).max(-1)
    return out, size, most


def attend_bound(out, size, most, dim, keys):
    """How far a kernel with exact bf16 products, fp32 sums and weights rounded
    to bf16 may be from ``attend`` after its own rounding to bf16:

    * a score is a sum of dim products in fp32 and a few multiplications:
      off by at most d = (dim + 8) 2^-24 times the sum of the terms' sizes,
      and so is the running maximum; a weight by a factor within 1 +- 2.2 d;
    * exp2 in fp32 and the rescalings: at most 2^-20 of a weight in all (64
      tiles of rounding 2^-24, and 2^-22 of the exponential and its argument
      for each unit of the argument's size, which small weights have);
    * a weight rounds to bf16 (2^-8), the sums over the keys lose keys 2^-24 at most;
    * the result rounds to bf16 (2^-8 of itself, and the subnormals' 2^-134)."""
    d = (dim + 8) * 2.0 ** -24 * most[..., None]
    return (2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.2 * d + 2.0 ** -20 + 2.0 ** -22 * (1 + 2 * most[..., None])
                                      + 2 * keys * 2.0 ** -24) * 1.01 * size + 2.0 ** -130)
