"""GPU tests of wal_delta: rows past max_new are kept nowhere, in either form and in calls of both; calls of both forms whose
chunks take several launches.  Tolerances as in test_gpu_delta.py: states 1e-6 of their norm and the oracle's bounds, outputs
3e-3 of a sequence's norm."""
import numpy as np
import pytest

from oracle import blocks as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_delta import Case, host, recurrence  # noqa: E402


@pytest.fixture(scope="module")
def wal():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import ternary_hybrid_bit_amd as w
    return w


@pytest.mark.parametrize("new,max_new,kw", [
    ([3, 5], 2, {}), ([5, 0, 9], 4, dict(dk=128, dv=64)), ([130, 70], 60, {}), ([130, 70], 64, dict(dk=128)), ([200, 65, 3], 65, dict(raw=False)),
    ([300, 10], 129, dict(dk=128, dv=96)), ([1, 2, 90, 1], 70, {}), ([1, 30, 100, 1, 1], 20, dict(dk=128, dv=64)), ([500] + [1] * 40, 100, {}),
    ([24] * 40, 9, dict(kh=4, group=2)), ([40] + [9, 1, 0] * 16, 30, dict(kh=8, group=2, dv=64)), ([300] + [1, 3] * 70, 200, dict(kh=8, group=2, dv=64)),
])
def test_rows_past_max_new_are_kept_nowhere(wal, new, max_new, kw):
    c = Case(wal, new, seed=max_new, max_new=max_new, **kw)
    print(f"delta new={new[:9]} max_new={max_new}", flush=True)
    out, state = c.call()
    heads = lambda t, d: host(t).reshape(c.n, t.shape[1] // d, d)  # noqa: E731
    q, k, v = heads(c.q, c.dk), heads(c.k, c.dk), heads(c.v, c.dv)
    alpha, beta = B.gates(host(c.a), host(c.b), *(None if t is None else host(t) for t in (c.decay, c.shift)))
    want = host(c.state0)
    for s, (a, m) in enumerate(zip(c.starts, new)):
        e = a + min(m, max_new)
        ref, want, _, err = B.delta(q[a:e], k[a:e], v[a:e], alpha[a:e], beta[a:e], [0, e - a], want, [c.slots[s]], c.desc.norm_eps,
                                    c.desc.scale, 2.0 ** -16)
        assert (out[e:a + m] == -7).all(), s
        got, kept = host(out[a:e]).reshape(ref.shape), host(state)[c.slots[s]]
        assert np.linalg.norm(got - ref) <= 3e-3 * np.linalg.norm(ref), s
        if m:
            gap = kept - want[c.slots[s]]
            assert (np.sqrt((gap ** 2).sum(1)) <= err[c.slots[s]]).all(), s
            assert np.linalg.norm(gap) <= 1e-6 * np.linalg.norm(want[c.slots[s]]), s
    others = [i for i in range(c.places) if i not in c.slots or not new[list(c.slots).index(i)]]
    assert torch.equal(state[others], c.state0[others])


@pytest.mark.parametrize("new,kw", [
    ([1, 1, 300, 1, 8, 0, 1] + [1] * 20, dict(dk=128, dv=64, kh=8, group=3)), ([200] + [1] * 40, dict(dk=128, kh=16, group=2)),
    ([8, 9, 1] * 9 + [70], dict(kh=8, group=4, dv=96)), ([1, 130] + [2, 0] * 20, dict(keep=False, kh=16, group=1, dv=64)),
    ([1] * 130 + [24, 16, 17, 100], dict(kh=8, group=4)), ([1] * 33 + [70, 2], dict(before=6, behind=5, kh=4, group=4, dv=64)),
    ([1, 1, 80] + [3] * 30, dict(slots=[40, 1, 0] + list(range(2, 32)), places=33, kh=8, group=2, dv=64)),
    ([30] + [0] * 40 + [20], dict(kh=8, group=4)), ([32, 1, 5, 17] + [2, 25, 16] * 5, dict(kh=16, group=4, dv=128)),   # (the last all token by token)
])
def test_prompts_among_single_tokens_of_many_heads(wal, new, kw):
    """From 1024 slices of states on each sequence of such a call goes in its own form."""
    c = Case(wal, new, seed=len(new) + 190, **kw)
    assert len(new) * c.h * (c.dv // 32) >= 1024 and c.n - c.before <= max(new) + (len(new) - 1) * 16
    c.check()


def test_both_forms_and_several_launches(wal):
    """A long prompt among single tokens: more chunks than one launch's share of the workspace."""
    new = [1] * 50 + [5000] + [1] * 40
    c = Case(wal, new, kh=96, group=1, dk=128, dv=32, seed=84)
    assert c.ws.numel() < (c.n // 64 + len(new)) * 96 * 50000 / 2   # three launches or more
    out, state = (t.clone() for t in c.call())
    ref, ref_state = recurrence(c)
    for s in range(len(new)):
        rows = slice(int(c.starts[s]), int(c.starts[s + 1]))
        assert (out[rows].double() - ref[rows]).norm() <= 3e-3 * ref[rows].norm(), s
        got, want = state[c.slots[s]].double(), ref_state[c.slots[s]]
        assert (got - want).norm() <= 1e-6 * want.norm(), s
    again, state2 = c.call()
    assert torch.equal(again, out) and torch.equal(state2, state)
