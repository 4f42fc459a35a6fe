"""GPU tests of wal_delta where values of a column differ widely in size, and of every output of calls on chunks, against
the recurrence in float64 (oracle/blocks.py).

Tolerances, fixed before the first run.  States: the oracle's bounds with the steps of test_gpu_delta.py, 2^-18 a token and
2^-16 on chunks.  Outputs, each element: 2^-8 of the value (its rounding to bf16) and the oracle's bound with a step of
* 2^-18 token by token;
* 2^-14 on chunks: what an output sees enters its products as two parts in bf16, so a term x y is off by 3 2^-18 of itself
  (each factor 2^-18, and the product of the second parts is left out), a row u that a token stores is at most
  2 (|v| + |s|) as long as beta is at most 2, which makes 6 2^-18, Q S one more 2^-18, sums of 64 and 128 terms in fp32
  2 2^-18, and the states' own 2^-16: 13 2^-18 in all.
Where keys point along axes every element of a state is made of its own row's writes alone, and the zeros of a key add
exact zeros: each is within 2^-18 of itself then, and each output within 2^-8 + 2^-14 of itself."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_delta import Case, host  # noqa: E402

STEP_STATE, STEP_OUT = 2.0 ** -16, 2.0 ** -14


@pytest.fixture(scope="module")
def wal():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import ternary_hybrid_bit_amd as w
    return w


def check_each(c):
    """Every output and every column of the states within its own bound: (outputs, what they should be)."""
    print(f"delta new={c.new[:9]} {c.kh}/{c.h} heads {c.dk}x{c.dv}", flush=True)
    chunked = c.ws.numel() > 16
    out, state = c.call()
    ref, ref_state, _, err_state = c.oracle(STEP_STATE if chunked else 2.0 ** -18)
    _, _, err, _ = c.oracle(STEP_OUT if chunked else 2.0 ** -18)
    rows = slice(c.before, int(c.starts[-1]))
    got, ref, err = host(out).reshape(ref.shape)[rows], ref[rows], err[rows]
    off = np.abs(got - ref)
    assert (off <= err + 2.0 ** -8 * np.abs(ref)).all(), (off / (err + 2.0 ** -8 * np.abs(ref))).max()
    if c.keep:
        gap = np.sqrt(((host(state) - ref_state) ** 2).sum(2))
        assert (gap <= err_state).all(), (gap[err_state > 0] / err_state[err_state > 0]).max()
    return got, ref


def put(t, rows, cols, value):
    t[rows, cols] = torch.as_tensor(value, dtype=t.dtype, device="cuda")


@pytest.mark.parametrize("new,kw", [
    ([17], {}), ([64], dict(dk=128, dv=128)), ([63, 64, 65, 1, 0, 128], dict(dk=128, dv=96)), ([300], dict(kh=1, group=4, raw=False)),
    ([1, 2, 70, 33], dict(keep=False)), ([90, 31], dict(norm=False, dk=128, dv=64)), ([500], dict(kh=1, group=1, dk=128, dv=256, scale=0.3)),
    ([129, 40], dict(before=5, behind=70, dk=128)),
])
def test_every_output_of_prompts(wal, new, kw):
    check_each(Case(wal, new, seed=len(new) + 150, **kw))


@pytest.mark.parametrize("beta", [0.5, 1.0, 2.0, None])
@pytest.mark.parametrize("new,dk", [([7, 5], 128), ([200, 70], 128), ([130], 64)])
def test_keys_alike_and_steps_up_to_two(wal, new, dk, beta):
    """Keys of cosines of about 0.9 (stored rows alternate and cancel), steps over the whole range (None: from 1 to 2): each output
    within its bound, and all of them no further off than their rounding to bf16 makes them, to a tenth (which
    products of 11 bits pass: 2.1e-3 to 3.2e-3 for 1.66e-3)."""
    c = Case(wal, new, kh=2, group=2, dk=dk, dv=64, raw=False, seed=71)
    rng = np.random.default_rng(72)
    kw = c.kh * dk
    k = rng.standard_normal(kw) + 0.33 * rng.standard_normal((c.n, kw))
    c.k.copy_(torch.from_numpy(k.astype(np.float32)).cuda())
    c.a.copy_(torch.from_numpy((-0.01 * rng.random((c.n, c.h))).astype(np.float32)).cuda())
    b = rng.uniform(1, 2, (c.n, c.h)) if beta is None else np.full((c.n, c.h), beta)
    c.b.copy_(torch.from_numpy(b.astype(np.float32)).cuda())
    got, ref = check_each(c)
    rounded = torch.from_numpy(ref).to(torch.bfloat16).double().numpy()
    if sum(new) > 20:
        assert np.linalg.norm(got - ref) <= 1.1 * np.linalg.norm(rounded - ref)


@pytest.mark.parametrize("new", [[8, 6], [64, 10], [150, 70]])
@pytest.mark.parametrize("ratio", [1e3, 1e6, 1e9, 1e12, 1e30])
def test_a_large_row_that_is_forgotten(wal, new, ratio):
    """One row of v much larger than the others and a decay of nothing at the token behind it: what follows is exact again, and
    what came before was so all along.  In other columns the large row lies elsewhere, and is not forgotten."""
    c = Case(wal, new, kh=2, group=2, dk=64, dv=64, raw=False, seed=81)
    p = min(new) // 2
    for s in range(len(new)):
        at = int(c.starts[s]) + p
        c.v[at, :32] *= ratio
        c.v[at + 1, 32:64] *= ratio
        c.v[at:at + 3, 64:] *= ratio
        put(c.a, at + 1, 0, -1e30)
        put(c.a, slice(at + 3, at + 4), 1, -200.0)
    check_each(c)


@pytest.mark.parametrize("new", [[8, 6], [100, 70]])
@pytest.mark.parametrize("ratio", [1e6, 1e12, 1e30])
def test_a_large_row_after_small_ones(wal, new, ratio):
    """Nothing is forgotten: the rows before a large one keep their bits, also in the same chunk."""
    c = Case(wal, new, kh=1, group=2, dk=128, dv=32, raw=False, seed=82)
    for s in range(len(new)):
        c.v[int(c.starts[s + 1]) - 2] *= ratio
    check_each(c)


@pytest.mark.parametrize("new", [[8, 6], [64, 70]])
@pytest.mark.parametrize("ratio", [1e4, 1e8, 1e12])
def test_a_large_state_that_decays(wal, new, ratio):
    """States far larger than what a call stores, gone within a few tokens or within a chunk."""
    c = Case(wal, new, kh=2, group=1, dk=128, dv=64, raw=False, seed=83)
    c.state0 *= ratio
    c.a[:, 0] = -6.0 if max(new) < 10 else -1.2
    put(c.a, int(c.starts[0]) + 2, 1, -np.inf)
    put(c.a, int(c.starts[1]) + 2, 1, -np.inf)
    check_each(c)


@pytest.mark.parametrize("new", [[8, 7], [128, 60]])
@pytest.mark.parametrize("ratio", [1.0, 1e6, 1e12, 1e30, None])
def test_keys_along_axes(wal, new, ratio):
    """A state is a table then: a row of it that is much larger than the others takes nothing from them (None: as large as
    bf16 holds)."""
    c = Case(wal, new, kh=1, group=2, dk=64, dv=32, raw=False, norm=False, seed=84)
    rng = np.random.default_rng(85)
    c.state0 *= 0.0
    c.k.zero_()
    c.q.zero_()
    rows = torch.arange(c.n, device="cuda")
    axis = torch.from_numpy(rng.integers(0, 64, c.n)).cuda()
    read = torch.from_numpy(rng.integers(0, 64, c.n)).cuda()
    for s in range(len(new)):
        a, e = int(c.starts[s]), int(c.starts[s + 1])
        axis[a + 1], axis[a + 2] = 5, 9
        axis[a + 3:e][axis[a + 3:e] == 5] = 6     # row 5 is written once, and large
        read[a + 2:e:2] = axis[a + 2:e:2]
        c.v[a + 1] = 3.38e38 if ratio is None else c.v[a + 1] * ratio
    c.k[rows, axis] = 1.0
    c.q[rows, read] = 1.0
    c.b.fill_(1.0)
    c.a.zero_()
    out, state = c.call()
    ref, ref_state, _, _ = c.oracle(0.0)
    got = host(out).reshape(ref.shape)
    assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -14) * np.abs(ref)).all()
    assert (np.abs(host(state) - ref_state) <= 2.0 ** -18 * np.abs(ref_state)).all()


@pytest.mark.parametrize("new", [[9, 5], [17, 30]])
def test_steps_far_past_two(wal, new):
    """beta |k|^2 = 20 enlarges a state up to 19 times a token: what stays inside fp32's range is finite in both forms."""
    c = Case(wal, new, kh=1, group=2, dk=64, dv=32, raw=False, norm=False, seed=86)
    c.k.mul_(float(np.sqrt(10.0)) / c.k.float().norm(dim=1, keepdim=True).clamp_min(1e-3))
    c.b.fill_(2.0)
    c.a.fill_(0.0)
    _, ref_state, _, _ = c.oracle(0.0)
    assert np.abs(ref_state).max() < 1e38
    out, state = c.call()
    assert torch.isfinite(out).all() and torch.isfinite(state).all()
