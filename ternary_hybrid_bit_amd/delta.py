"""A layer of the gated delta rule over packed matrices: the products, the causal
convolution of q | k | v, the delta rule on the sequences' states, the gated norm
of its heads and the o product.

``DeltaLayer`` is the shortest complete use of wal_conv, wal_delta and wal_head_norm with a gate, as
``attention.AttentionLayer`` is of the attention: forward() takes the new tokens of
any sequences, whole prompts, chunks of them and single tokens alike.
examples/delta_layer.py runs one.
"""
from __future__ import annotations

from typing import Sequence

import numpy as np

from . import (WAL_MAX_BATCH, _norm_weight, _types, _vec, make_delta_desc, wal_conv, wal_delta,
               wal_delta_workspace_size, wal_gemm_prefill, wal_gemm_small, wal_head_norm, wal_prefill_workspace_size,
               wal_workspace_size)
from .attention import _counts, _sequences


def _check_small(conv, conv_bias, decay, shift, norm, eps: float, channels: int, value_heads: int, value_dim: int, device):
    """Everything that wal_conv, wal_delta and wal_head_norm would refuse of a layer's small tensors."""
    T = _types()
    for name, t in (("conv", conv), ("conv_bias", conv_bias), ("decay", decay), ("shift", shift), ("norm", norm)):
        if t is None and name == "conv_bias":
            continue
        if not isinstance(t, T.tensor):
            raise TypeError(f"{name} must be a torch tensor on the GPU, not {type(t).__name__}")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the matrices on {device}")
        if t.data_ptr() % (16 if name.startswith("conv") else t.element_size()):
            raise ValueError(f"{name} is not aligned to {16 if name.startswith('conv') else t.element_size()} bytes")
    if conv.dtype not in T.acts:
        raise TypeError(f"conv has dtype {conv.dtype}; expected one of {[str(d) for d in T.acts]}")
    if conv.dim() != 2 or conv.shape[0] != channels or not 2 <= conv.shape[1] <= 4 or not conv.is_contiguous():
        raise ValueError(f"conv must be contiguous, [{channels}][2 to 4 taps] (shape {tuple(conv.shape)})")
    if conv_bias is not None:
        _norm_weight(T, conv_bias, "conv_bias", channels)
        if conv_bias.dtype is not conv.dtype:
            raise TypeError(f"conv_bias has dtype {conv_bias.dtype}, conv {conv.dtype}: they must be the same")
    _vec(T, decay, "decay", T.f32, value_heads)
    _vec(T, shift, "shift", T.f32, value_heads)
    _norm_weight(T, norm, "norm", value_dim)
    if not 2.0 ** -126 <= eps < float("inf"):
        raise ValueError(f"eps {eps}: normal, finite and above 0")


class DeltaLayer:
    """qkv, z, ab, o: (info, packed bytes on the GPU) of the layer's matrices.  qkv has key_heads heads of key_dim for
    q, as many for k and value_heads heads of value_dim for v, one after another, z as many rows as v, ab two for each
    value head (what the decays are made of, then the steps).  conv [channels of qkv][taps] and conv_bias (or None): the
    convolution; decay, shift fp32 [value_heads]: the gates' (wal_delta); norm [value_dim]: the weight of the outputs'
    norm, with eps.  States are kept for max_seqs sequences."""

    def __init__(self, qkv, z, ab, o, conv, decay, shift, norm, key_heads: int, value_heads: int, key_dim: int,
                 value_dim: int, max_seqs: int, conv_bias=None, eps: float = 1e-6, norm_eps: float = 1e-6):
        import torch
        self.torch, self.dev = torch, qkv[1].device
        self.mats = (qkv, z, ab, o)
        # all here, so that no call is refused between the launches that change states
        _check_small(conv, conv_bias, decay, shift, norm, eps, 2 * key_heads * key_dim + value_heads * value_dim, value_heads,
                     value_dim, self.dev)
        self.conv, self.conv_bias, self.decay, self.shift, self.norm, self.eps = conv, conv_bias, decay, shift, norm, eps
        self.desc = make_delta_desc(key_heads, value_heads, key_dim, value_dim, norm_eps=norm_eps)
        wal_delta_workspace_size(self.desc, 1, 1, 1)   # refuses heads and sizes that wal_delta does not take
        kw, vw = key_heads * key_dim, value_heads * value_dim
        self.parts = (slice(0, kw), slice(kw, 2 * kw), slice(2 * kw, 2 * kw + vw))
        for name, m, rows in (("qkv", qkv, 2 * kw + vw), ("z", z, vw), ("ab", ab, 2 * value_heads)):
            if m[0].d.out != rows:
                raise ValueError(f"{name} has {m[0].d.out} rows; {key_heads} key heads of {key_dim} and {value_heads} "
                                 f"value heads of {value_dim} need {rows}")
        if o[0].d.in_ != vw:
            raise ValueError(f"o has {o[0].d.in_} columns; {value_heads} value heads of {value_dim} need {vw}")
        # the products' type: a prompt cut anywhere gives the convolution the same rows
        self.rows = torch.zeros((max_seqs, conv.shape[1] - 1, 2 * kw + vw), device=self.dev)
        self.state = torch.zeros((max_seqs, value_heads, key_dim, value_dim), device=self.dev)
        self.ws = {}

    def _workspace(self, what: str, n: int):
        """A zeroed buffer for the products, whose first words they keep zero between calls, and others."""
        if what not in self.ws or self.ws[what].numel() < n:
            self.ws[what] = self.torch.zeros(max(n, 16), dtype=self.torch.uint8, device=self.dev)
        return self.ws[what]

    def _product(self, m, X, Y=None):
        """X W^T; with Y None only what it needs is made: its output, and its workspace."""
        info, W = m
        small = X.shape[0] <= WAL_MAX_BATCH
        ws = self._workspace("product" if small else "prompt",
                             (wal_workspace_size if small else wal_prefill_workspace_size)(info, X.shape[0]))
        if Y is None:
            return self.torch.empty((X.shape[0], info.d.out), device=self.dev)
        return (wal_gemm_small if small else wal_gemm_prefill)(info, W, X, Y, ws=ws)

    def release(self, s: int):
        """Sequence s is done: the next tokens of that number begin a new one."""
        s, = _sequences([s], self.state.shape[0])
        self.rows[s].zero_()
        self.state[s].zero_()

    def _run(self, X, new, slots):
        """forward() and prompt().  wal_conv and wal_delta change the kept rows and the states; what they and the calls behind
        them could refuse is checked before, here or by the constructor."""
        torch = self.torch
        QKV, Z, AB = (self._product(m, X, self._product(m, X)) for m in self.mats[:3])
        h, n = self.desc.value_heads, X.shape[0]
        fused = torch.empty(QKV.shape, dtype=torch.bfloat16, device=self.dev)
        out = torch.empty((n, Z.shape[1]), dtype=torch.bfloat16, device=self.dev)
        Y = self._product(self.mats[3], out)
        ws = self._workspace("delta", wal_delta_workspace_size(self.desc, len(new), n, max(new)))
        starts = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=self.dev)
        rows = state = None
        if slots is not None:
            rows, state, slots = self.rows, self.state, torch.tensor(slots, dtype=torch.int32, device=self.dev)
        wal_conv(QKV, self.conv, starts, fused, state=rows, slots=slots, bias=self.conv_bias)
        q, k, v = (fused[:, p] for p in self.parts)
        wal_delta(self.desc, q, k, v, AB[:, :h], AB[:, h:], starts, out, state=state, slots=slots, ws=ws,
                  decay=self.decay, shift=self.shift, max_new=max(new))
        wal_head_norm(out, out, self.norm, self.desc.value_dim, eps=self.eps, gate=Z)
        return self._product(self.mats[3], out, Y)

    def forward(self, X, seqs: Sequence[int], new: Sequence[int]):
        """X bf16 [n][hidden] -> fp32 [n][hidden]: new[i] tokens of sequence seqs[i] each, one after another, taken
        into the sequences' states."""
        new = _counts(new, X)
        return self._run(X, new, _sequences(seqs, self.state.shape[0], new))

    def prompt(self, X, lens: Sequence[int]):
        """The same for whole prompts whose states are not kept (scoring)."""
        return self._run(X, _counts(lens, X), None)


def packed_delta_layer(seed: int, hidden: int, key_heads: int, value_heads: int, key_dim: int, value_dim: int, taps: int = 4,
                       rank: int = 16):
    """Random packed qkv, z, ab, o of a layer and its small tensors, on the GPU, as DeltaLayer takes them."""
    import torch

    import synth

    from . import pack_matrix
    kw, vw, out = key_heads * key_dim, value_heads * value_dim, []
    for i, (rows, cols) in enumerate([(2 * kw + vw, hidden), (vw, hidden), (2 * value_heads, hidden), (hidden, vw)]):
        blob, info = pack_matrix(synth.make_matrix(seed, i, rows, cols, k=8, n_paths=1, rank=rank))
        out.append((info, torch.from_numpy(blob).to("cuda")))
    g = np.random.default_rng(seed)
    step = np.exp(g.uniform(np.log(1e-3), np.log(0.1), value_heads))
    small = (0.5 * g.standard_normal((2 * kw + vw, taps)), g.uniform(1, 16, value_heads), np.log(np.expm1(step)),
             1 + 0.3 * g.standard_normal(value_dim))
    return out + [torch.from_numpy(np.asarray(t, np.float32)).to("cuda") for t in small]
