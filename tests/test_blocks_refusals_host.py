"""More of what the binding and the library's calls of the blocks take and refuse, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import ternary_hybrid_bit_amd as wal
from test_blocks_host import F32, I32, I64, meta

ARG, SHAPE, BUFFER, ALIGN = -1, -2, -5, -6


def test_rows_whose_elements_lie_apart():
    """Refused where there are rows; tensors without any have the strides that their maker gave them (numpy: 0)."""
    assert torch.from_numpy(np.zeros((0, 256), np.float32)).stride() == (0, 0)
    w = meta(64, dt=F32)
    for rows, error in ((0, "GPU"), (1, "unit stride"), (3, "unit stride")):
        far, near = meta(rows, 256, stride=(512, 0)), meta(rows, 256)
        pos, turns = meta(rows, dt=I32), meta(32, dt=I64)
        for call in (lambda: wal.wal_head_norm(far, near, w, 64), lambda: wal.wal_head_norm(near, far, w, 64),
                     lambda: wal.wal_rope(far, near, pos, turns, 64)):
            with pytest.raises(ValueError, match=error):
                call()


# ---- the delta rule's workspace ----------------------------------------------------
# Addresses are made up: every call is refused before any launch, or has nothing to do.

FAR, APART = 1 << 44, 1 << 36
NAMES = ("q", "k", "v", "a", "b", "de", "sh", "starts", "state", "slots", "out", "ws")
SIZES = (2, 4, 64, 32, 1e-6, 0.125)


def delta(n, new, need, seqs=1, **kw):
    p = dict(dict({name: FAR + i * APART for i, name in enumerate(NAMES)}, wsb=need), **kw)
    return wal._lib.wal_delta(ctypes.byref(wal.wal_delta_desc(*SIZES)), p["q"], 128, p["k"], 128, p["v"], 128, p["a"], 4, p["b"], 4,
                              p["de"], p["sh"], p["starts"], seqs, n, new, p["state"], p["slots"], 2, p["out"], 128, p["ws"],
                              p["wsb"], None)


def size_of(n, new, seqs=1, sizes=SIZES):
    need = ctypes.c_size_t(1)
    assert wal._lib.wal_delta_workspace_size(ctypes.byref(wal.wal_delta_desc(*sizes)), seqs, n, new, ctypes.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("n,new,seqs", [(64, 64, 1), (300, 70, 5), (1 << 20, 1 << 20, 1)])   # the last in several launches
def test_delta_workspace_refusals(n, new, seqs):
    need = size_of(n, new, seqs)
    assert need > 0
    at = {name: FAR + i * APART for i, name in enumerate(NAMES)}
    go = lambda **kw: delta(n, new, need, seqs, **kw)  # noqa: E731
    assert go(ws=None) == ARG
    assert go(wsb=need - 1) == BUFFER and go(wsb=0) == BUFFER
    for off in (2, 16, 128):
        assert go(ws=at["ws"] + off, wsb=need + 256) == ALIGN
    for name in NAMES[:-1]:
        assert go(ws=at[name]) == ARG, name                       # begins with it
        assert go(ws=at[name] - (need - 1) // 256 * 256) == ARG, name   # its last bytes are the other's first
    assert delta(0, new, 0, seqs, ws=None) == 0   # nothing to do and none needed


def test_delta_workspace_sizes():
    assert size_of(8, 8) == 0 and size_of(0, 64) == 0 and size_of(64, 64, seqs=0) == 0 and size_of(64, 0) == 0
    assert size_of(9, 9) > 0
    # chunks of 64 rows, one more for each sequence's part of one; never above what a launch's share and two states need
    one, two = size_of(64, 64), size_of(640, 640)
    assert one < two <= 8 * one
    sizes = (16, 48, 128, 128, 1e-6, 0.125)
    longest = size_of(1 << 24, 1 << 24, sizes=sizes)
    assert longest == size_of(1 << 20, 1 << 20, sizes=sizes) < (256 << 20) + 2 * 4 * 48 * 128 * 128 + (4 << 20)
    for bad in (((1 << 24) + 1, 64, 1), (64, (1 << 24) + 1, 1), (64, 64, (1 << 24) + 1)):
        need = ctypes.c_size_t()
        assert wal._lib.wal_delta_workspace_size(ctypes.byref(wal.wal_delta_desc(*SIZES)), bad[2], bad[0], bad[1],
                                                 ctypes.byref(need)) == SHAPE
    assert wal._lib.wal_delta_workspace_size(ctypes.byref(wal.wal_delta_desc(*SIZES)), 1, 64, 64, None) == ARG
