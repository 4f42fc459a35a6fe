"""Norms of single heads, the causal convolution and the gated delta rule in
float64, written from the formulas of include/wal.h (numpy only, nothing shared
with the library).

Each function also gives what its error bound is made of, so that a test states
its tolerance per element instead of choosing one.
"""
from __future__ import annotations

import numpy as np


def silu(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def head_norm(x, weight, eps):
    """x [n][heads][dim] over the root of each head's mean square, times weight."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def conv(x, weight, bias, starts, state, slots, use_silu):
    """x [n][channels], weight [channels][taps], state [places][taps - 1][channels] -> (out, the new state, sums of
    |w x| + |bias|).  Rows outside the sequences: NaN."""
    x, w, state = np.asarray(x, np.float64), np.asarray(weight, np.float64), np.array(state, np.float64)
    taps = w.shape[1]
    out, size = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    b = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, np.float64)
    for s, slot in enumerate(slots):
        a, e = starts[s], starts[s + 1]
        kept = 0 <= slot < state.shape[0]
        before = state[slot] if kept else np.zeros((taps - 1, x.shape[1]))
        rows = np.concatenate([before, x[a:e]])
        for t in range(a, e):
            part = rows[t - a:t - a + taps] * w.T
            y = part.sum(0) + b
            out[t] = silu(y) if use_silu else y
            size[t] = np.abs(part).sum(0) + np.abs(b)
        if kept and e > a:
            state[slot] = rows[len(rows) - (taps - 1):]
    return out, state, size


def conv_bound(out, size, taps, use_silu, bf16):
    """fp32 sums of taps products and a bias, one rounding each, of parts that add up to `size`; silu's slope is below
    1.1, its exponential, sum and quotient within 2^-21 of it; bf16 rounds by 2^-8 of the value."""
    err = (taps + 1) * 2.0 ** -24 * size
    if use_silu:
        err = 1.1 * err + 2.0 ** -21 * np.abs(out)
    return err + (2.0 ** -8 * np.abs(out) if bf16 else 0.0) + 1e-36


def gates(a, b, decay, shift):
    """(alpha, beta) from what a call is given."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    if decay is None:
        return np.exp(np.minimum(a, 0.0)), b
    with np.errstate(over="ignore"):
        return np.exp(-np.asarray(decay, np.float64) * np.logaddexp(a + shift, 0.0)), 1.0 / (1.0 + np.exp(-b))


def delta(q, k, v, alpha, beta, starts, state, slots, norm_eps, scale, step):
    """q, k [n][key heads][key_dim], v [n][value heads][value_dim], alpha, beta [n][value heads], state
    [places][value heads][key_dim][value_dim] -> (out, the new state, bounds of the two).

    Bounds: for a column s of a state with error E (2-norms) a token's exact step does not enlarge E, as long as |k| <= 1
    and 0 <= beta <= 2 (it multiplies it by alpha (1 - beta k k^T)); its arithmetic adds at most step (|v| + |s|):
    `step` stands for the roundings of the sums of a token, of a chunk of them where the call works on chunks."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    state = np.array(state, np.float64)
    group = v.shape[1] // k.shape[1]
    if norm_eps > 0:
        q, k = (t / np.sqrt((t * t).sum(-1, keepdims=True) + norm_eps) for t in (q, k))
    q, k = np.repeat(q, group, 1), np.repeat(k, group, 1)
    out, out_err = np.full(v.shape, np.nan), np.full(v.shape, np.nan)
    err_state = np.zeros((state.shape[0], state.shape[1], state.shape[3]))
    for s, slot in enumerate(slots):
        kept = 0 <= slot < state.shape[0]
        m = state[slot].copy() if kept else np.zeros(state.shape[1:])
        err = np.zeros((state.shape[1], state.shape[3]))
        for t in range(starts[s], starts[s + 1]):
            size = np.abs(v[t]) + np.sqrt((m * m).sum(1))
            m = alpha[t][:, None, None] * m
            u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", m, k[t]))
            m = m + k[t][:, :, None] * u[:, None, :]
            err = np.abs(alpha[t])[:, None] * err + step * size
            qn = np.sqrt((q[t] * q[t]).sum(-1, keepdims=True))
            out[t] = scale * np.einsum("hkv,hk->hv", m, q[t])
            out_err[t] = abs(scale) * qn * (err + step * np.sqrt((m * m).sum(1)))
        if kept and starts[s + 1] > starts[s]:
            state[slot], err_state[slot] = m, err
    return out, state, out_err, err_state
