"""The attention layer's page lists without a GPU: the launches are recorded instead of made."""
import types

import numpy as np
import pytest
import torch

from ternary_hybrid_bit_amd import attention

QH, KVH, D, PAGE = 4, 2, 64, 16


def matrix(out):
    return types.SimpleNamespace(d=types.SimpleNamespace(out=out)), torch.zeros(1, dtype=torch.uint8)


@pytest.fixture
def calls(monkeypatch):
    """Keyword arguments of each wal_kv_write and wal_attn_paged: slots, pos and lens, starts, tables as lists."""
    got = []
    monkeypatch.setattr(attention, "wal_kv_write", lambda d, cache, slots, K, V, pos, **kw: got.append(
        dict(slots=slots.tolist(), pos=pos.tolist())))

    def attn(d, cache, tables, lens, starts, q, out, ws, **kw):
        got[-1].update(tables=tables.tolist(), lens=lens.tolist(), starts=starts.tolist(), **kw)
        return out
    monkeypatch.setattr(attention, "wal_attn_paged", attn)
    return got


def layer(n_pages, max_seqs):
    return attention.AttentionLayer(matrix(QH * D), matrix(KVH * D), matrix(KVH * D), matrix(256), D, n_pages, max_seqs,
                                    page_size=PAGE)


def rows(n, k=None, v=None):
    return tuple(torch.zeros((m, h * D)) for m, h in ((n, QH), (n if k is None else k, KVH), (n if v is None else v, KVH)))


def state(a):
    return list(a.free), [list(p) for p in a.pages], list(a.lens)


def test_tokens_go_to_their_pages(calls):
    a = layer(6, 3)
    assert a.attend(*rows(23), [2, 0], [20, 3]).shape == (23, QH * D)
    a.attend(*rows(14), [0, 1], [14, 0])
    assert a.lens == [17, 0, 20] and [len(p) for p in a.pages] == [2, 0, 2] and len(a.free) == 2
    assert len({*a.free, *sum(a.pages, [])}) == 6
    first, second = calls
    p2, p0 = a.pages[2], a.pages[0]
    assert first["slots"] == [p2[j // PAGE] * PAGE + j % PAGE for j in range(20)] + [p0[0] * PAGE + j for j in range(3)]
    assert first["pos"] == [*range(20), *range(3)] and first["lens"] == [20, 3] and first["starts"] == [0, 20, 23]
    assert (first["max_new"], first["max_len"]) == (20, 20)
    assert second["slots"] == [p0[j // PAGE] * PAGE + j % PAGE for j in range(3, 17)] and second["lens"] == [17, 0]
    assert second["tables"][0][:2] == p0 and second["starts"] == [0, 14, 14]
    a.release(2)
    assert a.lens[2] == 0 and a.pages[2] == [] and sorted(a.free + p0) == list(range(6))


def test_running_out_of_pages_changes_nothing(calls):
    """The call raises before it changes anything, so that a caller may release a sequence and try again."""
    a = layer(4, 4)
    a.attend(*rows(5), [3], [5])
    before = state(a)
    with pytest.raises(RuntimeError, match="page"):
        a.attend(*rows(64), [0, 1, 2], [16, 16, 32])          # four pages, three free
    assert state(a) == before and len(calls) == 1
    a.release(3)
    a.attend(*rows(64), [0, 1, 2], [16, 16, 32])
    assert a.lens == [16, 16, 32, 0] and not a.free
    assert calls[1]["pos"] == [*range(16), *range(16), *range(32)] and len(set(calls[1]["slots"])) == 64
    before = state(a)
    with pytest.raises(RuntimeError, match="page"):
        a.attend(*rows(1), [0], [1])
    assert state(a) == before


def test_a_failing_launch_changes_nothing(monkeypatch):
    a = layer(4, 2)
    before = state(a)
    with pytest.raises(ValueError, match="GPU"):              # the binding's own check: the tensors are on the CPU
        a.attend(*rows(20), [0], [20])
    assert state(a) == before
    monkeypatch.setattr(attention, "wal_kv_write", lambda *args, **kw: None)
    with pytest.raises(ValueError, match="GPU"):
        a.attend(*rows(20), [0], [20])
    assert state(a) == before
    # the last product of forward() too: its tokens are not counted
    monkeypatch.setattr(attention, "wal_attn_paged", lambda *args, **kw: args[6])

    def product(m, X):
        if m is a.mats[3]:
            raise MemoryError
        return torch.zeros((X.shape[0], m[0].d.out))
    monkeypatch.setattr(a, "_product", product)
    with pytest.raises(MemoryError):
        a.forward(torch.zeros((20, 256)), [0], [20])
    assert state(a) == before


@pytest.mark.parametrize("seqs,new,n", [
    ([0, 0], [2, 3], (5,)),                # a sequence twice: its first rows would see its last tokens
    ([0, 1], [5], (5,)), ([0], [3, 2], (5,)),
    ([0], [6], (5,)), ([0], [4], (5,)),    # counts and rows
    ([0], [5], (5, 4)), ([0], [5], (5, 5, 6)), ([0], [5], (4, 5, 5)),
    ([0, 1], [6, -1], (5,)), ([2], [5], (5,)), ([-1], [5], (5,)), ([], [], (0,)),
])
def test_refusals(calls, seqs, new, n):
    a = layer(8, 2)
    before = state(a)
    with pytest.raises(ValueError):
        a.attend(*rows(*n), seqs, new)
    assert state(a) == before and not calls


def test_refusals_of_other_calls(monkeypatch):
    a = layer(8, 2)
    with pytest.raises(TypeError):
        a.attend(*rows(5), [0], [5.0])
    for s in (-1, 2):
        with pytest.raises(ValueError):
            a.release(s)
    monkeypatch.setattr(a, "_product", lambda m, X: torch.zeros((X.shape[0], m[0].d.out)))
    for lens in ([], [4], [6], [6, -1]):
        with pytest.raises(ValueError, match="tokens|prompt"):
            a.prompt(torch.zeros((5, 256)), lens)
    assert state(a) == ([*range(8)], [[], []], [0, 0])


def test_counts_may_be_numpy_numbers(calls):
    a = layer(8, 2)
    a.attend(*rows(5), np.array([1, 0]), np.array([2, 3]))
    assert a.lens == [3, 2]
