"""GPU tests of wal_delta against the recurrence in float64 (oracle/blocks.py).

Tolerances, fixed before the first run: the bounds that the oracle carries along, with for a token's arithmetic
* 2^-18 (|v| + |s|) of a column s (2-norms) in calls of few tokens: a product with k or q adds up key_dim / 32 terms in a
  thread and the threads' in 7 steps, 11 roundings of 2^-24 of sums that |k| <= 1 bounds by |s|, and 6 more for the norms'
  factors; the gates' exponentials and logarithms are off by 2^-20 (alpha log(alpha) is below 0.37); the update's own two
  roundings: below 2^-18 in all;
* 2^-16 in calls on chunks of 64 tokens: sums of up to 64 such terms meet once more, 64 roundings of 2^-24 of terms with
  weights of at most 1;
* bf16 output: 2^-8 of the value, and on chunks what the rounded operands of the products that only outputs see are off by
  (half precision is within what bf16 would be):
  2^-7 (|s| + the largest |v|) of a row's own sums, in place of which the relative 2-norm of all outputs is held to 3e-3,
  too (1.7e-3 is what rounding the exact outputs to bf16 gives).
"""
import numpy as np
import pytest

from oracle import blocks as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


class Case:
    """Inputs of a call, and the oracle's answer."""

    def __init__(self, wal, new, kh=2, group=2, dk=64, dv=32, raw=True, norm=True, seed=1, slots=None, places=None, before=0,
                 behind=0, keep=True, scale=None, max_new=None):
        rng = np.random.default_rng(seed)
        self.wal, self.new, self.h, self.kh, self.dk, self.dv, self.keep = wal, list(new), kh * group, kh, dk, dv, keep
        self.desc = wal.make_delta_desc(kh, self.h, dk, dv, norm_eps=1e-6 if norm else 0.0, scale=scale)
        self.starts = before + np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.before, self.n = before, int(self.starts[-1]) + behind
        self.max_new = max(1, max(new)) if max_new is None else max_new
        kw, vw, h = kh * dk, self.h * dv, self.h
        x = rng.standard_normal((self.n, 2 * kw + vw)) * np.exp(0.3 * rng.standard_normal(2 * kw + vw))
        x = x / (1 + np.exp(-x))
        if not norm:
            x[:, :2 * kw] *= dk ** -0.5   # of about the size that keys without a norm have to have: |k| below 1
            for j in range(kh):
                part = x[:, kw + j * dk:kw + (j + 1) * dk]
                part /= np.maximum(1.01 * np.sqrt((part * part).sum(1, keepdims=True)), 1.0)
        fused = torch.from_numpy(x.astype(np.float32)).cuda().to(torch.bfloat16)
        self.q, self.k, self.v = fused[:, :kw], fused[:, kw:2 * kw], fused[:, 2 * kw:]
        g = rng.standard_normal((self.n, 2 * h + 3))
        self.decay = self.shift = None
        if raw:
            step = np.exp(rng.uniform(np.log(1e-3), np.log(0.1), h))
            self.shift = torch.from_numpy(np.log(np.expm1(step)).astype(np.float32)).cuda()
            self.decay = torch.from_numpy(rng.uniform(1, 16, h).astype(np.float32)).cuda()
        else:
            g[:, :h] = -0.1 * np.exp(g[:, :h])
            g[:, h:] = 1 / (1 + np.exp(-g[:, h:]))
        g = torch.from_numpy(g.astype(np.float32)).cuda()
        self.a, self.b = g[:, :h], g[:, h:2 * h]
        self.places = places or len(self.new) + 2
        self.slots = rng.permutation(self.places)[:len(self.new)] if slots is None else np.asarray(slots)
        self.state0 = torch.from_numpy((0.2 * rng.standard_normal((self.places, h, dk, dv))).astype(np.float32)).cuda()
        self.ws = torch.full((max(wal.wal_delta_workspace_size(self.desc, len(self.new), self.n, self.max_new), 16),), 255,
                             dtype=torch.uint8, device="cuda")

    def call(self, state=None, out=None, starts=None):
        self.state = (self.state0.clone() if state is None else state) if self.keep else None
        self.out = torch.full((self.n, self.h * self.dv + 8), -7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        self.wal.wal_delta(self.desc, self.q, self.k, self.v, self.a, self.b, i32(self.starts if starts is None else starts),
                           self.out[:, :self.h * self.dv], state=self.state, slots=i32(self.slots) if self.keep else None,
                           ws=self.ws, decay=self.decay, shift=self.shift, max_new=self.max_new)
        torch.cuda.synchronize()
        return self.out[:, :self.h * self.dv], self.state

    def oracle(self, step):
        heads = lambda t, d: host(t).reshape(self.n, t.shape[1] // d, d)  # noqa: E731
        alpha, beta = B.gates(host(self.a), host(self.b), *(None if t is None else host(t) for t in (self.decay, self.shift)))
        return B.delta(heads(self.q, self.dk), heads(self.k, self.dk), heads(self.v, self.dv), alpha, beta, self.starts,
                       host(self.state0) if self.keep else np.zeros((0, self.h, self.dk, self.dv)),
                       self.slots if self.keep else [-1] * len(self.new), self.desc.norm_eps, self.desc.scale, step)

    def check(self):
        print(f"delta new={self.new[:9]} {self.kh}/{self.h} heads {self.dk}x{self.dv} places={self.places}", flush=True)
        chunked = self.ws.numel() > 16
        out, state = self.call()
        ref, ref_state, err, err_state = self.oracle(2.0 ** -16 if chunked else 2.0 ** -18)
        rows = slice(self.before, int(self.starts[-1]))
        got, ref, err = host(out).reshape(ref.shape)[rows], ref[rows], err[rows]
        off = np.abs(got - ref)
        if chunked:
            size = np.abs(host(self.v)).max() * 1.0 + np.sqrt((ref_state ** 2).sum(2)).max(initial=0.0)
            assert (off <= err + 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * size).all()
            if ref.size:
                assert np.linalg.norm(off) <= 3e-3 * np.linalg.norm(ref)
        else:
            assert (off <= err + 2.0 ** -8 * np.abs(ref)).all()
        if self.keep:
            gap = np.sqrt(((host(state) - ref_state) ** 2).sum(2))   # of each column
            assert (gap <= err_state).all()
            if ref.size:
                moved = host(self.state0) != ref_state
                assert np.linalg.norm((host(state) - ref_state)[moved]) <= 1e-6 * np.linalg.norm(ref_state[moved])
        assert (self.out[:self.before] == -7).all() and (self.out[int(self.starts[-1]):] == -7).all()
        assert (self.out[:, self.h * self.dv:] == -7).all()
        return self


@pytest.mark.parametrize("new,kw", [
    ([1], {}), ([1], dict(kh=16, group=3, dk=128, dv=128)), ([1] * 5, dict(dk=128, dv=256)), ([1] * 70, dict(kh=1, group=1, raw=False)),
    ([2, 0, 5, 1, 0], dict(dv=96)), ([0, 0], {}), ([5, 3, 4], dict(dk=128, dv=64, norm=False)), ([16, 9, 2], dict(kh=3, group=1, raw=False)),
    ([24, 1] + [3] * 62, dict(kh=2, group=2, dv=64)), ([7, 8], dict(kh=1, group=5, dk=128, dv=192)),
    ([1, 1, 1], dict(slots=[-1, 9, 1], places=4)), ([3, 2], dict(keep=False)), ([4, 1], dict(before=3, behind=5)),
    ([2, 2], dict(scale=-0.7, dv=160)),
])
def test_few_tokens(wal, new, kw):
    Case(wal, new, seed=len(new), **kw).check()


@pytest.mark.parametrize("new,kw", [
    ([17], {}), ([64], dict(dk=128, dv=128)), ([65], {}), ([63, 64, 65, 1, 0, 128], dict(dk=128, dv=96)), ([300], dict(kh=1, group=4, raw=False)),
    ([1, 2, 70, 33], dict(keep=False)), ([200, 5], dict(slots=[7, -3], places=8)), ([129, 40], dict(before=5, behind=70, dk=128)),
    ([90, 31], dict(norm=False, dk=128, dv=64)), ([500], dict(kh=1, group=1, dk=128, dv=256, scale=0.3)), ([1000, 3, 70], dict(kh=1, group=2)),
])
def test_prompts(wal, new, kw):
    Case(wal, new, seed=len(new) + 50, **kw).check()


@pytest.mark.parametrize("new,kw", [
    ([1, 1, 300, 1, 8, 0, 1], dict(dk=128, dv=64)), ([200] + [1] * 40, dict(dk=128)), ([8, 9, 1], {}), ([1, 130], dict(keep=False)),
    ([1] * 70 + [24, 25, 100], dict(kh=2, group=2)), ([1, 2, 90, 1], dict(max_new=70, raw=False)), ([1, 70, 2], dict(before=6, behind=5)),
    ([1, 1, 80], dict(slots=[9, 1, 0], places=3)), ([30, 0, 0, 0, 0, 20], {}),
])
def test_prompts_among_single_tokens(wal, new, kw):
    """Each sequence of such a call goes in its own form."""
    c = Case(wal, new, seed=len(new) + 90, **kw)
    if "max_new" not in kw:
        c.check()
    else:   # what max_new cuts off is left
        out, _ = c.call()
        ref, *_ = c.oracle(0.0)
        for s, (a, k) in enumerate(zip(c.starts, new)):
            rows = slice(a, a + min(k, c.max_new))
            got, want = host(out[rows]).reshape(-1, c.h, c.dv), ref[rows]
            assert np.linalg.norm(got - want) <= 3e-3 * np.linalg.norm(want)
            assert (out[a + c.max_new:a + k] == -7).all()


@pytest.mark.parametrize("kh,group,dv", [(3, 4, 256), (3, 2, 32), (8, 2, 64), (1, 7, 256)])
def test_heads_side_by_side(wal, kh, group, dv):
    """Heads that share a key head on one chiplet, and by themselves: numbers of workgroups that leave chiplets uneven."""
    Case(wal, [70, 100, 90], kh=kh, group=group, dv=dv, seed=kh + dv).check()


@pytest.mark.parametrize("dk,dv", [(64, 32), (128, 128)])
def test_chunks_and_tokens_continue_each_other(wal, dk, dv):
    """A sequence taken in pieces of any size, through the state, stays with the oracle's bounds of the whole."""
    c = Case(wal, [150], dk=dk, dv=dv, seed=8)
    ref, ref_state, err, err_state = c.oracle(2.0 ** -16)
    state, slots = c.state0.clone(), i32(c.slots)
    at = 0
    for n in (70, 1, 1, 5, 64, 9):
        rows = slice(at, at + n)
        out = torch.empty((n, c.h * dv), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(wal.wal_delta_workspace_size(c.desc, 1, n, n), 16), dtype=torch.uint8, device="cuda")
        wal.wal_delta(c.desc, c.q[rows], c.k[rows], c.v[rows], c.a[rows], c.b[rows], i32([0, n]), out, state=state, slots=slots,
                      ws=ws, decay=c.decay, shift=c.shift, max_new=n)
        got = host(out).reshape(n, c.h, dv)
        assert np.linalg.norm(got - ref[rows]) <= 3e-3 * np.linalg.norm(ref[rows])
        at += n
    assert at == 150
    assert (np.sqrt(((host(state) - ref_state) ** 2).sum(2)) <= err_state).all()
    slot = c.slots[0]
    assert np.linalg.norm(host(state)[slot] - ref_state[slot]) <= 1e-6 * np.linalg.norm(ref_state[slot])


@pytest.mark.parametrize("new", [[4, 3], [150, 70]])
def test_gates_at_their_ends(wal, new):
    """Decays of nothing and of everything, steps of 0 and 1, in any order: no overflow, and what follows is exact again."""
    c = Case(wal, new, raw=False, seed=21)
    rng = np.random.default_rng(22)
    a = rng.choice([0.0, -1e-3, -0.5, -30.0, -200.0, -1e30, -np.inf, 3.0], (c.n, c.h))
    a[:, 1] = rng.choice([-1e-3, -300.0], c.n, p=[0.9, 0.1])       # a state thrown away now and then, kept well between
    c.a.copy_(torch.from_numpy(a.astype(np.float32)).cuda())
    c.b.copy_(torch.from_numpy(rng.choice([0.0, 1.0, 0.5], (c.n, c.h)).astype(np.float32)).cuda())
    c.check()


@pytest.mark.parametrize("new", [[4, 3], [150, 70]])
def test_equal_keys_and_missing_ones(wal, new):
    """The same key again and again (each token replaces what the one before stored), and keys and queries of zeros."""
    c = Case(wal, new, dk=128, dv=64, seed=31)
    c.k.copy_(c.k[:1].expand(c.n, -1))
    c.k[c.n // 2] = 0
    c.q[c.n // 3] = 0
    c.b.fill_(20.0)
    c.check()


@pytest.mark.parametrize("new", [[6, 5, 4], [100, 150, 70]])
@pytest.mark.parametrize("what", ["q", "k", "v", "a", "b"])
def test_non_finite_values(wal, new, what):
    """A NaN or infinity touches its own token and later ones of its own sequence and head (v: column), nothing before."""
    c = Case(wal, new, kh=2, group=1, dk=64, dv=64, seed=41)
    clean, clean_state = (t.clone() for t in c.call())
    row = int(c.starts[1]) + new[1] // 2 + 1
    t = getattr(c, what)
    width = {"q": 64, "k": 64, "v": 64, "a": 1, "b": 1}[what]
    t[row, width + (3 if width > 1 else 0)] = float("nan") if what in "ab" else float("inf")      # head 1
    out, state = c.call()
    bad = ~torch.isfinite(out).cpu().numpy()
    want = np.zeros_like(bad)
    end = int(c.starts[2])
    if what == "q":
        want[row, 64:128] = True
    elif what == "v":
        want[row:end, 64 + 3] = True
    else:
        want[row:end, 64:128] = True
    assert not (bad & ~want).any()
    assert bad[row:row + 1][want[row:row + 1]].all()
    if what != "q":
        assert bad[want].all()
    # a chunk's other columns, heads and sequences keep their bits
    same = torch.from_numpy(~want).cuda()
    assert torch.equal(out[same], clean[same])
    left = torch.isfinite(state).cpu().numpy()
    lost = np.zeros_like(left)
    if what == "v":
        lost[c.slots[1], 1, :, 3] = True
    elif what != "q":
        lost[c.slots[1], 1] = True
    assert np.array_equal(~left, lost)
    assert torch.equal(state[torch.from_numpy(~lost).cuda()], clean_state[torch.from_numpy(~lost).cuda()])


@pytest.mark.parametrize("new", [[3, 1, 7], [130, 64, 7]])
def test_repeated_calls_and_neighbours_rows(wal, new):
    """The same bits again, whatever the workspace and the rows outside the sequences hold."""
    c = Case(wal, new, dk=128, dv=64, seed=51, before=4, behind=9)
    out, state = (t.clone() for t in c.call())
    for t in (c.q, c.k, c.v, c.a, c.b):
        t[:4] = float("nan")
        t[c.n - 9:] = float("nan")
    c.ws.random_(0, 255)
    again, state2 = c.call()
    assert torch.equal(out, again) and torch.equal(state, state2)


@pytest.mark.parametrize("new", [[3, 5], [130, 70]])
def test_max_new_cuts_and_starts_that_do_not_rise(wal, new):
    c = Case(wal, new, seed=61, max_new=min(new) - 1)
    out, state = c.call()
    short = Case(wal, new, seed=61, max_new=min(new) - 1)
    ref, *_ = short.oracle(0.0)
    for s in (0, 1):
        a = int(c.starts[s])
        got = host(out[a:a + c.max_new]).reshape(c.max_new, c.h, -1)
        assert np.linalg.norm(got - ref[a:a + c.max_new]) <= 3e-3 * np.linalg.norm(ref[a:a + c.max_new])
        assert (out[a + c.max_new:int(c.starts[s + 1])] == -7).all()
    n = c.n
    for starts in ([n - 1, 1, n], [-5, 2, 10 ** 6], [2 ** 31 - 1, -2 ** 31, 7], [n + 3, n + 5, n + 9], [0, 0, 0]):
        whole = torch.full((n + 20, c.h * c.dv + 8), -7.0, dtype=torch.bfloat16, device="cuda")
        state = c.state0.clone()
        c.call(state=state, out=whole[10:n + 10], starts=starts)
        assert (whole[:10] == -7).all() and (whole[n + 10:] == -7).all() and (whole[:, c.h * c.dv:] == -7).all()
        others = [i for i in range(c.places) if i not in c.slots]
        assert torch.equal(state[others], c.state0[others])


def recurrence(c):
    """The definition in float64 with torch on the GPU, for calls that are long for numpy: (out, state)."""
    heads = lambda t, d: t.double().unflatten(1, (-1, d))  # noqa: E731
    q, k, v = heads(c.q, c.dk), heads(c.k, c.dk), heads(c.v, c.dv)
    q, k = ((t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(c.h // c.kh, 1) for t in (q, k))
    alpha, beta = (torch.from_numpy(t).cuda() for t in B.gates(host(c.a), host(c.b), host(c.decay), host(c.shift)))
    out, state = torch.zeros_like(v), c.state0.double()
    for s, slot in enumerate(c.slots):
        m = state[slot].clone()
        for t in range(c.starts[s], c.starts[s + 1]):
            m *= alpha[t][:, None, None]
            u = beta[t][:, None] * (v[t] - torch.matmul(k[t][:, None], m)[:, 0])
            m += k[t][:, :, None] * u[:, None]
            out[t] = c.desc.scale * torch.matmul(q[t][:, None], m)[:, 0]
        state[slot] = m
    return out.flatten(1), state


def test_calls_cut_into_several_launches(wal):
    """More chunks than one launch's share of the workspace: states of sequences that go on are carried over, short ones lie
    between and at the cuts."""
    new = [1500, 3, 64, 2500, 1, 700, 0, 130]
    c = Case(wal, new, kh=96, group=1, dk=128, dv=32, seed=81)
    assert c.ws.numel() < (c.n // 64 + len(new)) * 96 * 50000   # less than all chunks at once need
    out, state = c.call()
    ref, ref_state = recurrence(c)
    for s in range(len(new)):
        rows = slice(int(c.starts[s]), int(c.starts[s + 1]))
        assert (out[rows].double() - ref[rows]).norm() <= 3e-3 * ref[rows].norm(), s
        got, want = state[c.slots[s]].double(), ref_state[c.slots[s]]
        assert (got - want).norm() <= 1e-6 * want.norm(), s
    again, state2 = c.call()
    assert torch.equal(again, out) and torch.equal(state2, state)


def test_many_sequences_cut_into_several_launches(wal):
    """A launch looks at the sequences that can have a place in it only."""
    rng = np.random.default_rng(82)
    new = [int(x) for x in rng.integers(0, 70, 160)] + [70]
    c = Case(wal, new, kh=96, group=1, dk=128, dv=32, seed=83)
    assert c.ws.numel() < (c.n // 64 + len(new)) * 96 * 50000 / 2   # three launches or more
    out, state = c.call()
    ref, ref_state = recurrence(c)
    for s in range(len(new)):
        rows = slice(int(c.starts[s]), int(c.starts[s + 1]))
        assert (out[rows].double() - ref[rows]).norm() <= 3e-3 * ref[rows].norm(), s
        got, want = state[c.slots[s]].double(), ref_state[c.slots[s]]
        assert (got - want).norm() <= 1e-6 * want.norm(), s
    others = [i for i in range(c.places) if i not in c.slots]
    assert torch.equal(state[others], c.state0[others])


@pytest.mark.parametrize("new", [[5, 6], [90, 70]])
@pytest.mark.parametrize("what", ["q", "k"])
def test_squares_past_the_range_are_not_finite(wal, new, what):
    """A row of finite values whose squares add up past fp32 is lost with a sign of it, token by token and on chunks."""
    c = Case(wal, new, kh=2, group=1, dk=64, dv=32, seed=43)
    clean, clean_state = (t.clone() for t in c.call())
    row = int(c.starts[1]) + new[1] // 2
    getattr(c, what)[row, 64:128] = 3e18      # 64 times 9e36 is past 3.4e38
    out, state = c.call()
    end = row + 1 if what == "q" else int(c.starts[2])
    assert (~torch.isfinite(out[row:end, 32:])).all()
    lost = torch.zeros_like(out, dtype=torch.bool)
    lost[row:end, 32:] = True
    assert torch.equal(out[~lost], clean[~lost])
    assert torch.isfinite(state[c.slots[1], 1]).any().item() == (what == "q")
    assert torch.equal(state[c.slots[0]], clean_state[c.slots[0]])


def test_calls_at_the_same_time(wal):
    """Two streams, each with its own workspace and states."""
    cases = [Case(wal, new, dk=128, dv=64, seed=90 + i) for i, new in enumerate(([300, 20], [257], [2, 1, 3]))]
    want = [tuple(t.clone() for t in c.call()) for c in cases]
    starts, slots = [i32(c.starts) for c in cases], [i32(c.slots) for c in cases]
    states, outs = [c.state0.clone() for c in cases], [torch.full_like(c.out, -7.0) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, st, x, y, state, out in zip(cases, streams, starts, slots, states, outs):
            with torch.cuda.stream(st):
                state.copy_(c.state0)
                wal.wal_delta(c.desc, c.q, c.k, c.v, c.a, c.b, x, out[:, :c.h * c.dv], state=state, slots=y, ws=c.ws, decay=c.decay,
                              shift=c.shift, max_new=c.max_new)
        torch.cuda.synchronize()
        for (o, s), state, out, c in zip(want, states, outs, cases):
            assert torch.equal(out[:, :c.h * c.dv], o) and torch.equal(state, s)


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 70, 130]])
def test_under_graph_and_on_another_stream(wal, new):
    c = Case(wal, new, dk=128, dv=128, kh=2, group=3, seed=71)
    out, state = (t.clone() for t in c.call())
    starts, slots = i32(c.starts), i32(c.slots)
    mine, mine_state = torch.full_like(out, -7.0), c.state0.clone()

    def go():
        wal.wal_delta(c.desc, c.q, c.k, c.v, c.a, c.b, starts, mine, state=mine_state, slots=slots, ws=c.ws, decay=c.decay,
                      shift=c.shift, max_new=c.max_new)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(mine, out) and torch.equal(mine_state, state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    mine_state.copy_(c.state0)
    eager = c.state0.clone()
    for _ in range(3):
        c.v.copy_(c.v.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = c.call(state=eager)
        assert torch.equal(mine, want) and torch.equal(mine_state, eager)
