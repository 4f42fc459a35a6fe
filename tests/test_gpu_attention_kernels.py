"""The attention kernels that ordinary test sizes do not reach, against the float64 oracle: the one of 256 query
rows (eight wavefronts), which takes calls with tiles of rows for every compute unit, and the one of 17 to 32
rows with heads of 128.  The rule that chooses the first is asked of the library, so that these sizes are known to
reach it.  Helpers and tolerances are those of test_gpu_attention.py."""
import numpy as np
import pytest

from oracle import attention as A

from test_gpu_attention import BF16, INT8, Paged, dev, host, i32, t16, wal  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def reaches_256_rows(wal, n_seqs, n, max_new, group, heads, dim):  # noqa: F811
    """The library's own rule (wal::attn_tile_rows of csrc/wal_attn.h)."""
    return wal._lib["_ZN3wal14attn_tile_rowsEjjjjjj"](n_seqs, n, max_new, group, heads, dim) == 256


def paged(wal, seqs, shape, fmt, **kw):  # noqa: F811
    group, heads, dim, page = shape
    p = Paged(wal, seqs, group, heads, dim, page, fmt, **kw)
    assert reaches_256_rows(wal, len(seqs), p.Q.shape[0], p.max_new, group, heads, dim)
    return p


def twice(p, **kw):
    """A call's output; a second call, on other contents of output and workspace, gives the same bits."""
    a = p.call(**kw).clone()
    p.out.fill_(-5.0)
    assert torch.equal(a, p.call(**kw))
    return a


SHAPES = [(8, 32, 128, 16), (5, 48, 64, 64), (1, 128, 64, 256), (3, 64, 128, 32)]   # group, key/value heads, dim, page
CHUNKS = [[(300, 300)],
          [(7, 7), (64, 64), (100, 3), (1, 1), (0, 0), (65, 65), (3, 5), (0, 2), (200, 90)],   # rows before the first token
          [(1500, 100), (40, 40), (900, 60), (2000, 1)],                                       # cut contexts
          [(1600, 288)]]                                                                       # one cut context


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seqs", range(len(CHUNKS)))
def test_chunks(wal, fmt, shape, seqs):  # noqa: F811
    print(f"chunks {CHUNKS[seqs]} {shape} fmt={fmt}", flush=True)
    p = paged(wal, CHUNKS[seqs], shape, fmt, seed=60 + seqs, pad=16)
    p.check(twice(p))
    assert (p.out[:, p.Q.shape[1]:] == -5.0).all()
    cut = wal.wal_attn_paged_workspace_size(p.d, p.group * p.heads, len(p.seqs), p.Q.shape[0], p.max_new, p.max_len) > 0
    # the last case's items are 288 (two rounds of workgroups) with the first two shapes, 256 (one) with the others
    assert cut == (seqs == 2 or seqs == 3 and shape in SHAPES[:2])


@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (-0.3, 1.0), (40.0, 1.0)])
def test_scales(wal, scale, gain):  # noqa: F811
    p = paged(wal, [(300, 300)], SHAPES[1], BF16, seed=7, gain=gain)
    p.check(p.call(scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("shape", [(8, 64, 64, 16), (8, 40, 128, 16), (8, 40, 128, 64)])
def test_pages_outside_the_cache_are_left_out(wal, fmt, shape):  # noqa: F811
    p = paged(wal, [(200, 120), (40, 40)], shape, fmt, seed=9)
    page = shape[3]
    present = [np.ones(n, bool) for n, _ in p.seqs]
    bad = [(0, 0, -1), (0, 2, p.d.n_pages), (1, 0, -2 ** 31)] + [(0, 5, 2 ** 31 - 1), (0, 12, -1), (1, 1, -1), (1, 2, -1)] * (page == 16)
    for i, at, to in bad:
        p.tables[i, at] = to
        present[i][page * at:page * at + page] = False
    out = twice(p)
    p.check(out, present=present)              # the second sequence sees nothing: zeros
    assert (out[120:] == 0).all()


def spoil(p, at, k=None, v=None):
    """The key and value of one token again, with an element replaced: (index, value)."""
    K, V = (torch.from_numpy(x[at:at + 1].reshape(1, -1).astype(np.float32)).to(dev()) for x in (p.k, p.v))
    for t, e in ((K, k), (V, v)):
        if e is not None:
            t[0, e[0]] = e[1]
    p.wal.wal_kv_write(p.d, p.cache, p.slots[at:at + 1], K, V)


def check_spoilt(p, new, bad, what):
    """Rows of the first sequence that see token bad: not finite in the first key/value head (in element 3 of it);
    everything else finite."""
    got = host(p.call()).reshape(-1, p.heads, p.group, p.dim)
    n = p.seqs[0][0]
    sees = np.zeros(len(got), bool)
    sees[:new] = n - new + np.arange(new) >= bad
    rest = got[:, 1:]
    assert sees.any() and np.isfinite(rest).all() and np.isfinite(got[~sees]).all()
    own = got[sees, 0]
    assert np.isnan(own).all() if what == "k" else not np.isfinite(own[..., 3]).any()


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("shape", [(8, 64, 64, 16), (8, 40, 128, 32)])
@pytest.mark.parametrize("bad", [1, 69, 119])      # seen by all rows; by the later half; by the last row
def test_nan_and_infinity(wal, fmt, shape, bad):  # noqa: F811
    new = 100
    for what, kw in (("k", dict(k=(5, np.nan))), ("v", dict(v=(3, np.inf))), ("v", dict(v=(3, np.nan)))):
        p = paged(wal, [(120, new), (80, 60)], shape, fmt, seed=11)
        spoil(p, bad, **kw)
        check_spoilt(p, new, bad, what)


PROMPTS = [[300], [64, 1, 0, 63, 65, 2, 130], [400, 129, 31]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens", range(len(PROMPTS)))
def test_prompt(wal, causal, shape, lens):  # noqa: F811
    group, heads, dim, _ = shape
    lens = PROMPTS[lens]
    print(f"prompt {lens} {shape} causal={causal}", flush=True)
    rng = np.random.default_rng(sum(lens) + dim)
    starts = np.concatenate([[0], np.cumsum(lens)])
    total, qw, kw = int(starts[-1]), group * heads * dim, heads * dim
    assert reaches_256_rows(wal, len(lens), total, max(lens), group, heads, dim)
    wide = t16(rng.standard_normal((total, qw + 2 * kw + 8)))
    Q, K, V = wide[:, :qw], wide[:, qw:qw + kw], wide[:, qw + kw:qw + 2 * kw]
    out, again = (torch.full((total + 1, qw + 24), f, dtype=torch.bfloat16, device=dev()) for f in (77.0, -5.0))
    for o, f in ((out, 77.0), (again, -5.0)):
        wal.wal_attn_prompt(Q, K, V, i32(starts), o[:total, :qw], dim, max(lens), causal=causal)
        assert (o[total] == f).all() and (o[:, qw:] == f).all()
    assert torch.equal(out[:total, :qw], again[:total, :qw])
    got = host(out[:total, :qw]).reshape(total, -1, dim)
    q, k, v = (host(x).reshape(total, -1, dim) for x in (Q, K, V))
    for a, b in zip(starts[:-1], starts[1:]):
        last = np.arange(b - a) if causal else np.full(b - a, b - a - 1)
        ref, size, most = A.attend(q[a:b], k[a:b], v[a:b], last, dim ** -0.5)
        assert (np.abs(got[a:b] - ref) <= A.attend_bound(ref, size, most, dim, b - a)).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,heads", [(64, 64), (128, 40)])
@pytest.mark.parametrize("bad", [0, 100, 199])
def test_prompt_nan_and_infinity(wal, causal, dim, heads, bad):  # noqa: F811
    group, lens = 8, [200, 40]
    n = sum(lens)
    assert reaches_256_rows(wal, 2, n, max(lens), group, heads, dim)
    rng = np.random.default_rng(bad)
    Q, K, V = (t16(rng.standard_normal((n, h * dim))) for h in (group * heads, heads, heads))
    for which, value in (("k", np.nan), ("v", np.inf), ("v", np.nan)):
        k, v, out = K.clone(), V.clone(), torch.empty_like(Q)
        (k if which == "k" else v)[bad, 3] = value
        wal.wal_attn_prompt(Q, k, v, i32([0, 200, 240]), out, dim, 200, causal=causal)
        got = host(out).reshape(n, heads, group, dim)
        sees = np.arange(n) < 200
        if causal:
            sees &= np.arange(n) >= bad
        assert np.isfinite(got[:, 1:]).all() and np.isfinite(got[~sees]).all()
        assert np.isnan(got[sees, 0]).all() if which == "k" else not np.isfinite(got[sees, 0][..., 3]).any()


# ---- 17 to 32 rows for each key/value head, heads of 128: a few new tokens -----

FEW = [[(517, 5)], [(33, 8), (8, 8), (3, 5), (0, 2), (700, 7), (65, 1)],
       [(9001, 8)], [(2500, 6), (2100, 8)]]     # joined by a launch of its own; by the workgroup that ends last


def few(wal, seqs, group, heads, fmt, page=16, **kw):  # noqa: F811
    p = Paged(wal, seqs, group, heads, 128, page, fmt, **kw)
    assert 16 < p.max_new * group <= 32
    return p


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("group,heads,page", [(4, 8, 16), (4, 1, 256), (3, 2, 64)])
@pytest.mark.parametrize("seqs", range(len(FEW)))
def test_few_tokens(wal, fmt, group, heads, page, seqs):  # noqa: F811
    seqs = [(n, min(new * 4 // group + 1, 32 // group) if group < 4 and new > 4 else new) for n, new in FEW[seqs]]
    print(f"few {seqs} group={group} heads={heads} page={page} fmt={fmt}", flush=True)
    p = few(wal, seqs, group, heads, fmt, page, seed=70, pad=16)
    p.check(twice(p))
    assert (p.out[:, p.Q.shape[1]:] == -5.0).all()


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("bad", [1, 115, 119])
def test_few_tokens_nan_and_infinity(wal, fmt, bad):  # noqa: F811
    for what, kw in (("k", dict(k=(5, np.nan))), ("v", dict(v=(3, np.inf))), ("v", dict(v=(3, np.nan)))):
        p = few(wal, [(120, 8), (80, 5)], 4, 2, fmt, seed=11)
        spoil(p, bad, **kw)
        check_spoilt(p, 8, bad, what)


@pytest.mark.parametrize("fmt", [BF16, INT8])
def test_few_tokens_pages_outside_the_cache(wal, fmt):  # noqa: F811
    p = few(wal, [(200, 8), (40, 8)], 4, 2, fmt, seed=9)
    present = [np.ones(n, bool) for n, _ in p.seqs]
    for i, at, to in ((0, 0, -1), (0, 5, p.d.n_pages), (0, 12, 2 ** 31 - 1), (1, 0, -2 ** 31), (1, 1, -1), (1, 2, -1)):
        p.tables[i, at] = to
        present[i][16 * at:16 * at + 16] = False
    p.check(twice(p), present=present)


# ---- the same bits from the same call ------------------------------------------

@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("seqs,shape", [([(517, 1)], (4, 8, 128, 64)), ([(3000, 1), (40, 1), (1100, 1)], (4, 2, 128, 16)),
                                        ([(20011, 1)], (4, 2, 64, 64)), ([(700, 257), (129, 2)], (3, 2, 256, 32)),
                                        ([(4100, 90), (300, 60)], (4, 2, 64, 64))])
def test_calls_repeat_exactly(wal, fmt, seqs, shape):  # noqa: F811
    group, heads, dim, page = shape
    p = Paged(wal, seqs, group, heads, dim, page, fmt, seed=80)
    p.check(twice(p))
