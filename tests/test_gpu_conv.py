"""GPU tests of wal_conv against float64 (oracle/blocks.py, whose conv_bound is the tolerance of each element)."""
import numpy as np
import pytest

from oracle import blocks as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f": torch.float32, "b": torch.bfloat16}


@pytest.fixture(scope="module")
def wal():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import ternary_hybrid_bit_amd as w
    return w


def host(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


def gpu(x, t, pad=0):
    r = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=TYPES[t], device="cuda")
    r[:, :x.shape[1]] = torch.from_numpy(np.asarray(x, np.float32)).cuda().to(TYPES[t])
    return r[:, :x.shape[1]]


def check(wal, new, channels, taps, tin="f", tw="b", tout="b", bias=True, silu=True, pad=0, slots=None, places=None, before=0, behind=0, seed=1):
    """One call against the oracle: rows before the first and behind the last sequence, and places of no sequence, stay."""
    print(f"conv new={list(new)[:8]}.. channels={channels} taps={taps} {tin}{tw}->{tout} {bias} {silu} pad={pad}", flush=True)
    rng = np.random.default_rng(seed)
    starts = before + np.concatenate([[0], np.cumsum(new)])
    n = int(starts[-1]) + behind
    X = gpu(rng.standard_normal((n, channels)), tin, pad)
    w = gpu(rng.standard_normal((channels, taps)), tw)
    b = gpu(rng.standard_normal((1, channels)), tw)[0] if bias else None
    places = places or len(new) + 2
    slots = rng.permutation(places)[:len(new)] if slots is None else np.asarray(slots)
    state = torch.from_numpy(rng.standard_normal((places, taps - 1, channels)).astype(np.float32)).cuda().to(TYPES[tin])
    was = state.clone()
    whole = torch.full((n, channels + pad), -7.0, dtype=TYPES[tout], device="cuda")
    out = whole[:, :channels]
    wal.wal_conv(X, w, i32(starts), out, state=state, slots=i32(slots), bias=b, silu=silu)
    torch.cuda.synchronize()
    ref, new_state, size = B.conv(host(X), host(w), None if b is None else host(b), starts, host(was), slots, silu)
    inside = slice(before, n - behind)
    err = np.abs(host(out) - ref)[inside]
    assert (err <= B.conv_bound(ref, size, taps, silu, tout == "b")[inside]).all()
    assert np.array_equal(host(state), new_state)
    assert (whole[:before] == -7).all() and (whole[n - behind:] == -7).all() and (not pad or (whole[:, channels:] == -7).all())
    return X, w, b, out


@pytest.mark.parametrize("new,channels,kw", [
    ([1], 8, {}), ([1], 10240, {}), ([2], 64, dict(taps=2)), ([3], 136, dict(taps=3, tin="b")), ([4], 72, dict(tin="b", tw="f", tout="f")),
    ([1] * 64, 8192, {}), ([1] * 65, 40, dict(tin="b")), ([0, 1, 2, 3, 4, 5, 6, 0], 48, dict(tw="f")),
    ([0, 0, 0], 16, {}), ([0, 5, 0, 0, 1, 0], 24, dict(taps=3, silu=False)), ([7, 1, 33, 2, 64, 3, 129, 1, 1], 520, dict(tin="b", pad=8)),
    ([1000], 256, dict(taps=2, tout="f", tw="f")), ([515, 1, 2, 700], 1032, dict(bias=False)), ([31, 30, 34, 1, 1, 1, 29, 35], 2048, dict(tin="b", taps=4)),
    ([5], 16384 * 4, dict(tin="f")), ([300, 11], 12000, dict(tin="f", tout="f")), ([1] * 300, 16, dict(taps=3)),
])
def test_conv(wal, new, channels, kw):
    kw = dict(dict(taps=4), **kw)
    check(wal, new, channels, seed=len(new) + channels, **kw)


def test_many_rows_and_sequences(wal):
    rng = np.random.default_rng(9)
    check(wal, rng.integers(0, 9, 5000), 64, 4, tin="b", seed=3)          # two looks at the starts
    check(wal, [40000, 3, 2500], 264, 4, tin="f", seed=4)                 # long tiles
    check(wal, [16000, 1, 2, 15, 0, 17, 3, 17100], 1024, 4, tin="b", seed=5)   # the longest
    check(wal, [1, 2, 3, 1, 0, 2], 520, 4, tin="b", seed=6)               # a row each


def test_rows_outside_the_sequences(wal):
    check(wal, [5, 0, 40], 64, 4, before=37, behind=50)
    check(wal, [5, 1], 64, 4, tin="b", before=3, behind=1)


def test_places_outside_the_state_begin_with_zeros(wal):
    check(wal, [3, 40, 1, 2], 64, 4, slots=[-1, 5, 2, 2 ** 31 - 1], places=5)


def test_without_a_state(wal):
    x = np.random.default_rng(1).standard_normal((50, 64))
    X, w, out = gpu(x, "f"), gpu(x[:4].T, "f"), torch.empty((50, 64), device="cuda")
    wal.wal_conv(X, w, i32([0, 20, 50]), out, silu=False)
    ref, _, size = B.conv(host(X), host(w), None, [0, 20, 50], np.zeros((0, 3, 64)), [-1, -1], False)
    assert (np.abs(host(out) - ref) <= B.conv_bound(ref, size, 4, False, False)).all()


@pytest.mark.parametrize("t", ["f", "b"])
def test_cut_anywhere_gives_the_same_bits(wal, t):
    X = gpu(np.random.default_rng(2).standard_normal((200, 96)), t)
    w, slots = gpu(np.random.default_rng(3).standard_normal((96, 4)), "f"), i32([1])
    whole, state = torch.empty((200, 96), device="cuda"), torch.zeros((2, 3, 96), dtype=TYPES[t], device="cuda")
    wal.wal_conv(X, w, i32([0, 200]), whole, state=state, slots=slots)
    for cuts in ([1, 2, 3, 5, 60], [33, 34, 66, 199], list(range(1, 200))):
        parts, again = torch.empty_like(whole), torch.zeros_like(state)
        for a, b in zip([0] + cuts, cuts + [200]):
            wal.wal_conv(X[a:b], w, i32([0, b - a]), parts[a:b], state=again, slots=slots)
        assert torch.equal(parts, whole) and torch.equal(again, state)


def test_non_finite_rows_touch_their_own_window_and_sequence_only(wal):
    x = np.random.default_rng(4).standard_normal((60, 16))
    x[19, 3], x[30, 5], x[45, 7] = np.nan, np.inf, -np.inf
    X, w, out = gpu(x, "f"), torch.ones((16, 4), device="cuda"), torch.empty((60, 16), device="cuda")
    wal.wal_conv(X, w, i32([0, 20, 60]), out, silu=False)
    bad = np.zeros((60, 16), bool)
    bad[19, 3] = bad[30:34, 5] = bad[45:49, 7] = True
    assert np.array_equal(~np.isfinite(host(out)), bad)


def test_starts_that_do_not_rise_touch_nothing_outside(wal):
    X, w = torch.randn((40, 16), device="cuda"), torch.ones((16, 4), device="cuda")
    for starts in ([30, 10, 40], [-5, 20, 1000], [2 ** 31 - 1, -2 ** 31, 7], [50, 60, 70], [0, 0, 0]):
        whole = torch.full((60, 16), 3.0, device="cuda")
        state = torch.full((4, 3, 16), 2.0, device="cuda")
        wal.wal_conv(X, w, i32(starts), whole[10:50], state=state, slots=i32([1, 2]))
        torch.cuda.synchronize()
        assert (whole[:10] == 3).all() and (whole[50:] == 3).all() and (state[0] == 2).all() and (state[3] == 2).all()


def test_under_graph(wal):
    X, w = torch.randn((5, 512), device="cuda"), torch.randn((512, 4), device="cuda").to(torch.bfloat16)
    state, starts, slots = torch.zeros((9, 3, 512), device="cuda"), i32(range(6)), i32([4, 2, 0, 7, 8])
    out = torch.empty((5, 512), dtype=torch.bfloat16, device="cuda")
    wal.wal_conv(X, w, starts, out, state=state.clone(), slots=slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wal.wal_conv(X, w, starts, out, state=state, slots=slots)
    state.zero_()
    mine, want = state.clone(), torch.empty_like(out)
    for _ in range(4):
        X.copy_(torch.randn((5, 512), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        wal.wal_conv(X, w, starts, want, state=mine, slots=slots)
        assert torch.equal(out, want) and torch.equal(state, mine)
