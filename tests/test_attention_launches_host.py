"""Attention calls of more workgroups than a launch takes are refused before any launch, without a GPU: such a launch would
do a part of the call only, without an error.  Addresses are made up: nothing is read."""
import ctypes

import pytest

import ternary_hybrid_bit_amd as wal

SHAPE = -2
FAR = 1 << 44


@pytest.mark.parametrize("max_new,n", [(1, 100), (40, 1 << 17)])   # few rows, and tiles of many
@pytest.mark.parametrize("n_seqs", [1 << 16, 1 << 20, 1 << 24])
def test_paged(n_seqs, max_new, n):
    d, need = wal.make_kv_desc(2, 16, 256, 64), ctypes.c_size_t()
    assert wal._lib.wal_attn_paged_workspace_size(ctypes.byref(d), 256, n_seqs, n, max_new, 16, ctypes.byref(need)) == 0
    assert wal._lib.wal_attn_paged(
        ctypes.byref(d), FAR, FAR + (1 << 30), 1, FAR + (1 << 31), FAR + (1 << 32), n_seqs, n, max_new, 16, FAR + (1 << 38),
        256, 256 * 64, 0.125, FAR + (1 << 40), 256 * 64, FAR + (1 << 43), need.value, None) == SHAPE


@pytest.mark.parametrize("n_seqs", [1 << 16, 1 << 20, 1 << 24])
def test_prompt(n_seqs):
    n = 1 << 17
    assert wal._lib.wal_attn_prompt(FAR, 256 * 64, FAR + (1 << 38), 256 * 64, FAR + (1 << 39), 256 * 64, FAR + (1 << 32), n_seqs, n, n,
                                    256, 256, 64, 0.125, 1, FAR + (1 << 40), 256 * 64, None) == SHAPE
