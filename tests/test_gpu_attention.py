"""GPU tests of the attention operators (wal_rope, wal_kv_write, wal_kv_read,
wal_attn_paged, wal_attn_prompt) against the float64 oracle (oracle/attention.py).

Tolerances, fixed before the first run:

* rotation, fp32 out: |err| <= 2^-21 m (|a| + |b|) (sine and cosine within
  2^-23 of fp32 polynomials on an exactly reduced angle, its conversion and
  constant 2^-23.5, three roundings of 2^-24); bf16 out: 2^-8 of the value more;
* int8 rows without a rotation: codes and scales equal to the definition's fp32
  arithmetic; with one: half a step of the row's scale and the rotation's bound;
* bf16 rows: the value rounded to nearest even;
* attention: per element, oracle/attention.py::attend_bound.
"""
import numpy as np
import pytest

from oracle import attention as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, INT8 = 0, 1


@pytest.fixture(scope="module")
def wal():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import ternary_hybrid_bit_amd as w
    return w


def dev():
    return torch.device("cuda:0")


def t16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dev()).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device=dev())


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def padded(x, pad, dtype):
    """x on the GPU inside rows that are pad wider, NaN around it."""
    t = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=dtype, device=dev())
    t[:, :x.shape[1]] = torch.from_numpy(np.asarray(x, np.float32)).to(dev()).to(dtype)
    return t


def table(wal, rot, scaling, factor):
    code = {"plain": 0, "linear": 1, "ntk": 2, "parts": 3}[scaling]
    turns, m = wal.wal_rope_freqs(wal.make_rope_desc(rot, 1e6, code, factor, 4096.0))
    f, _ = A.rope_freqs(rot, 1e6, scaling, factor, 4096.0)
    return torch.from_numpy(turns).to(dev()), f, m


# ---- rotation --------------------------------------------------------------

@pytest.mark.parametrize("n,heads,dim,rot,layout,scaling,tin,tout,pad", [
    (1, 32, 128, 128, 0, "plain", "f", "b", 0),
    (1, 1, 16, 16, 1, "plain", "f", "f", 0),
    (3, 40, 128, 96, 1, "parts", "b", "b", 1024),
    (37, 5, 64, 32, 0, "linear", "b", "f", 8),
    (130, 3, 80, 48, 0, "ntk", "f", "f", 4),
    (5, 2, 512, 512, 1, "plain", "b", "b", 0),
    (2111, 13, 256, 224, 0, "parts", "f", "b", 64),
    (4097, 10, 64, 64, 1, "plain", "b", "f", 0),
])
def test_rope(wal, n, heads, dim, rot, layout, scaling, tin, tout, pad):
    print(f"rope n={n} heads={heads} dim={dim} rot={rot} layout={layout} {scaling} {tin}->{tout}", flush=True)
    rng = np.random.default_rng(n + dim)
    types = {"f": torch.float32, "b": torch.bfloat16}
    turns, f, m = table(wal, rot, scaling, 1.0 if scaling == "plain" else 4.0)
    pos = rng.integers(0, 1 << 20, n)
    pos[0] = 2 ** 31 - 1 if n > 1 else 4097
    if n > 2:
        pos[1], pos[2] = -5, -2 ** 31
    X = padded(rng.standard_normal((n, heads * dim)), pad, types[tin])
    out = torch.full((n, heads * dim + pad), float("nan"), dtype=types[tout], device=dev())
    wal.wal_rope(X[:, :heads * dim], out[:, :heads * dim], i32(pos), turns, dim, layout=layout, magnitude=m)
    torch.cuda.synchronize()
    x = host(X[:, :heads * dim]).reshape(n, heads, dim)
    # the table's frequencies, not the unrounded ones: at position 2^31 half a unit of 2^-64 turns is 2^-34 turns
    f = turns.cpu().numpy().astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    # positions of 2^31 in float64: p f is off by 2^-53 p f, at most 2^-22 turns; reduce in integers instead
    frac = ((pos[:, None].astype(object) * turns.cpu().numpy().astype(object)[None]) % 2 ** 64)
    ang = np.array(frac, dtype=np.float64) * 2.0 ** -64 * 2 * np.pi
    ref, size = np.empty_like(x), np.empty_like(x)
    for i in range(n):
        r, s = A.rope(x[i:i + 1], [1.0], ang[i], m, layout == 1)
        ref[i], size[i] = r[0], s[0]
    got = host(out[:, :heads * dim]).reshape(n, heads, dim)
    bound = 2.0 ** -21 * size + (2.0 ** -8 * np.abs(ref) if tout == "b" else 0.0)
    assert (np.abs(got - ref) <= bound).all()
    if pad:
        assert torch.isnan(out[:, heads * dim:]).all()


@pytest.mark.parametrize("dtype", ["b", "f"])
def test_rope_in_place_equals_out_of_place(wal, dtype):
    t = torch.bfloat16 if dtype == "b" else torch.float32
    turns, _, m = table(wal, 64, "plain", 1.0)
    X = torch.randn((301, 6 * 128), device=dev()).to(t)
    pos, out = i32(np.arange(301)), torch.empty_like(X)
    wal.wal_rope(X, out, pos, turns, 128)
    wal.wal_rope(X, X, pos, turns, 128)
    assert torch.equal(X, out)


# ---- the cache --------------------------------------------------------------

def planes(wal, d, cache):
    f = wal.wal_kv_size(d)
    shape = (d.n_pages, d.kv_heads, d.page_size, d.head_dim)
    n = int(np.prod(shape))
    if d.fmt == BF16:
        got = [cache[o:o + 2 * n].view(torch.bfloat16).view(shape) for o in (f.off_k, f.off_v)]
        return got + [None, None]
    got = [cache[o:o + n].view(torch.int8).view(shape) for o in (f.off_k, f.off_v)]
    return got + [cache[o:o + 4 * n // d.head_dim].view(torch.float32).view(shape[:3]) for o in (f.off_ks, f.off_vs)]


def new_cache(wal, d, fill=0x7F):
    return torch.full((wal.wal_kv_size(d).total_bytes,), fill, dtype=torch.uint8, device=dev())


@pytest.mark.parametrize("n,heads,dim,page,tin", [(1, 1, 64, 16, "f"), (37, 8, 128, 16, "f"), (301, 5, 128, 64, "b"),
                                                 (70, 2, 256, 256, "f"), (4000, 8, 128, 32, "b")])
def test_int8_rows_equal_the_definition(wal, n, heads, dim, page, tin):
    print(f"int8 rows n={n} heads={heads} dim={dim} page={page} {tin}", flush=True)
    rng = np.random.default_rng(n)
    d = wal.make_kv_desc(-(-n // page) + 2, page, heads, dim, INT8)
    cache = new_cache(wal, d)
    before = cache.clone()
    k, v = (rng.standard_normal((n, heads * dim)) * np.exp(rng.standard_normal((n, 1)) * 3) for _ in range(2))
    if n > 30:
        k[3], v[4] = 0.0, 1e-35                  # held as zeros
        k[5, 7], v[6, 2], v[8, 0] = np.inf, np.nan, -np.inf
        k[9] *= 1e30 / np.abs(k[9]).max()
    slots = rng.permutation(d.n_pages * page)[:n].astype(np.int64)
    dropped = np.zeros(n, bool)
    if n > 30:
        slots[10], slots[11], slots[12] = -1, d.n_pages * page, 2 ** 31 - 1
        dropped[10:13] = True
    t = torch.float32 if tin == "f" else torch.bfloat16
    K, V = padded(k, 16, t), padded(v, 0, t)
    wal.wal_kv_write(d, cache, i32(slots), K[:, :heads * dim], V)
    pk, pv, ks, vs = planes(wal, d, cache)
    live = slots[~dropped]
    for X, plane, scales in ((K[:, :heads * dim], pk, ks), (V, pv, vs)):
        codes, scale = A.int8_rows(X.float().cpu().numpy().reshape(n, heads, dim))
        got, gs = plane.cpu().numpy()[live // page, :, live % page], scales.cpu().numpy()[live // page, :, live % page]
        assert np.array_equal(got, codes[~dropped]) and np.array_equal(gs, scale[~dropped], equal_nan=True)
    # nothing else was written
    keep = np.ones(d.n_pages * page, bool)
    keep[live] = False
    rest = np.nonzero(keep)[0]
    for a, b in zip(planes(wal, d, cache), planes(wal, d, before)):
        assert np.array_equal(a.cpu().view(torch.int8).numpy().reshape(*a.shape[:3], -1)[rest // page, :, rest % page],
                              b.cpu().view(torch.int8).numpy().reshape(*b.shape[:3], -1)[rest // page, :, rest % page])
    # read back
    for to in (torch.float32, torch.bfloat16):
        K2, V2 = (torch.full((n, heads * dim + 8), 7.0, dtype=to, device=dev()) for _ in range(2))
        wal.wal_kv_read(d, cache, i32(slots), K2[:, :heads * dim], V2[:, :heads * dim])
        for X, Y in ((K[:, :heads * dim], K2), (V, V2)):
            codes, scale = A.int8_rows(X.float().cpu().numpy().reshape(n, heads, dim))
            with np.errstate(invalid="ignore"):
                want = torch.from_numpy(codes.astype(np.float32) * scale[..., None])
            want[dropped] = 0.0
            assert torch.equal(Y[:, :heads * dim].cpu().nan_to_num(12345.0),
                               want.reshape(n, -1).to(to).nan_to_num(12345.0))
            assert (Y[:, heads * dim:] == 7.0).all()


@pytest.mark.parametrize("n,qh,heads,dim,rot,layout,page,tin", [(1, 32, 8, 128, 128, 0, 16, "f"),
                                                              (37, 4, 4, 64, 32, 1, 16, "b"),
                                                              (129, 10, 2, 256, 224, 0, 128, "f"),
                                                              (3001, 12, 3, 128, 96, 1, 64, "f")])
@pytest.mark.parametrize("fmt", [BF16, INT8])
def test_write_with_rotation(wal, n, qh, heads, dim, rot, layout, page, tin, fmt):
    print(f"write n={n} q={qh} kv={heads} dim={dim} rot={rot} layout={layout} page={page} {tin} fmt={fmt}", flush=True)
    rng = np.random.default_rng(n + fmt)
    d = wal.make_kv_desc(-(-n // page) + 1, page, heads, dim, fmt)
    cache = new_cache(wal, d)
    turns, f, m = table(wal, rot, "parts", 2.0)
    t = torch.float32 if tin == "f" else torch.bfloat16
    wide = torch.from_numpy(rng.standard_normal((n, (qh + 2 * heads) * dim)).astype(np.float32)).to(dev()).to(t)
    Q, K, V = wide[:, :qh * dim], wide[:, qh * dim:(qh + heads) * dim], wide[:, (qh + heads) * dim:]
    pos, slots = rng.integers(0, 50000, n), rng.permutation(d.n_pages * page)[:n]
    q_out = torch.empty((n, qh * dim), dtype=torch.bfloat16, device=dev())
    wal.wal_kv_write(d, cache, i32(slots), K, V, pos=i32(pos), turns=turns, layout=layout, magnitude=m, Q=Q,
                     Q_out=q_out)
    K2, V2 = (torch.empty((n, heads * dim), device=dev()) for _ in range(2))
    wal.wal_kv_read(d, cache, i32(slots), K2, V2)
    cut = lambda x: host(x).reshape(n, -1, dim)  # noqa: E731
    ref, size = A.rope(cut(Q), pos, f, m, layout == 1)
    tiny = 2.0 ** -21 * size + 1e-9 * size      # the oracle's unrounded frequencies: 50000 2^-65 turns
    assert (np.abs(cut(q_out) - ref) <= tiny + 2.0 ** -8 * np.abs(ref)).all()
    ref, size = A.rope(cut(K), pos, f, m, layout == 1)
    tiny = (2.0 ** -21 + 1e-9) * size
    if fmt == BF16:
        assert (np.abs(cut(K2) - ref) <= tiny + 2.0 ** -8 * np.abs(ref)).all()
        assert torch.equal(V2, V.to(torch.bfloat16).float())
    else:
        top = (np.abs(ref) + tiny).max(-1, keepdims=True)
        # half a step, the division's roundings (x times a rounded 127 / a: 127 2^-23 of a step) and the scale's
        assert (np.abs(cut(K2) - ref) <= top / 127 * (0.5 + 2.0 ** -15) + tiny + 2.0 ** -22 * np.abs(ref)).all()
        codes, scale = A.int8_rows(V.float().cpu().numpy().reshape(n, heads, dim))
        assert np.array_equal(V2.cpu().numpy().reshape(n, heads, dim), codes.astype(np.float32) * scale[..., None])
    assert torch.equal(K, wide[:, qh * dim:(qh + heads) * dim])


def test_write_q_in_place_in_a_fused_buffer(wal):
    n, d = 9, wal.make_kv_desc(2, 16, 2, 64, BF16)
    turns, _, m = table(wal, 64, "plain", 1.0)
    wide = torch.randn((n, 8 * 64), device=dev()).to(torch.bfloat16)
    q, k, v = wide[:, :256], wide[:, 256:384], wide[:, 384:]
    kv = wide[:, 256:].clone()
    want, c1, c2 = torch.empty((n, 256), dtype=torch.bfloat16, device=dev()), new_cache(wal, d), new_cache(wal, d)
    pos, slots = i32(np.arange(n) + 77), i32(np.arange(n) * 3)
    wal.wal_kv_write(d, c1, slots, k, v, pos=pos, turns=turns, magnitude=m, Q=q, Q_out=want)
    wal.wal_kv_write(d, c2, slots, k, v, pos=pos, turns=turns, magnitude=m, Q=q, Q_out=q)
    assert torch.equal(q, want) and torch.equal(c1, c2) and torch.equal(wide[:, 256:], kv)


def test_read_one_plane_and_nothing(wal):
    d = wal.make_kv_desc(4, 16, 2, 64, INT8)
    cache = new_cache(wal, d, 3)
    slots = i32([5, 63, 64, -7])
    K, V = (torch.full((4, 128), 9.0, device=dev()) for _ in range(2))
    wal.wal_kv_read(d, cache, slots, K, V)
    only = torch.full((4, 128), 9.0, device=dev())
    wal.wal_kv_read(d, cache, slots, V=only)
    assert torch.equal(only, V) and (V[2:] == 0).all() and (V[:2] != 0).all()
    wal.wal_kv_read(d, cache, slots, K=only)
    assert torch.equal(only, K)
    wal.wal_kv_read(d, cache, slots[:0], K=only[:0])
    wal.wal_kv_write(d, cache, slots[:0], K[:0], V[:0])


# ---- attention ----------------------------------------------------------------

class Paged:
    """Random sequences in a paged cache whose unused slots hold NaN (bf16) or NaN scales (int8)."""

    def __init__(self, wal, seqs, group, heads, dim, page, fmt, seed=0, pages=None, gain=1.0, pad=0):
        self.wal, self.seqs, self.dim, self.heads, self.group, self.page = wal, seqs, dim, heads, group, page
        rng = self.rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n, _ in seqs]
        self.d = d = wal.make_kv_desc(pages or sum(counts) + 2, page, heads, dim, fmt)
        self.cache = torch.full((wal.wal_kv_size(d).total_bytes,), 0xFF, dtype=torch.uint8, device=dev())
        order = (d.n_pages - 1 - rng.permutation(min(d.n_pages, sum(counts) + 2)))[:sum(counts)]
        self.tables = np.full((len(seqs), max(max(counts), 1) + 1), -1, np.int64)
        slots, at = [], 0
        for i, ((n, _), c) in enumerate(zip(seqs, counts)):
            self.tables[i, :c] = order[at:at + c]
            at += c
            j = np.arange(n)
            slots.append(self.tables[i][j // page] * page + j % page)
        total = sum(n for n, _ in seqs)
        self.bounds = np.concatenate([[0], np.cumsum([n for n, _ in seqs])])
        K, V = (torch.from_numpy((rng.standard_normal((total, heads * dim)) * g).astype(np.float32)).to(dev())
                for g in (gain, 1.0))
        self.slots = i32(np.concatenate(slots))
        if total:
            wal.wal_kv_write(d, self.cache, self.slots, K, V)
            wal.wal_kv_read(d, self.cache, self.slots, K, V)
        self.k, self.v = host(K).reshape(total, heads, dim), host(V).reshape(total, heads, dim)
        new = [m for _, m in seqs]
        self.starts = np.concatenate([[0], np.cumsum(new)])
        q = rng.standard_normal((self.starts[-1], group * heads * dim)) * gain
        self.Q = padded(q, pad, torch.bfloat16)[:, :q.shape[1]]
        self.out = torch.full(tuple(self.Q.shape[i] + (pad if i else 0) for i in (0, 1)), 77.0, dtype=torch.bfloat16,
                              device=dev())
        self.max_new, self.max_len = max(new + [1]), max([n for n, _ in seqs] + [1])

    def call(self, scale=None, stream=None, out=None, ws=None, slack=(0, 0)):
        w, d = self.wal, self.d
        out = self.out[:, :self.Q.shape[1]] if out is None else out
        new, most = self.max_new + slack[0], min(self.max_len + slack[1], self.tables.shape[1] * self.page)
        n = w.wal_attn_paged_workspace_size(d, self.group * self.heads, len(self.seqs), self.Q.shape[0], new, most)
        if ws is None:
            ws = torch.full((max(n, w.WAL_ATTN_WS_ZERO_BYTES),), 0xFF, dtype=torch.uint8, device=dev())
            ws[:w.WAL_ATTN_WS_ZERO_BYTES] = 0    # the rest must not matter
        self.ws = ws
        self.args = (i32(self.tables), i32([n for n, _ in self.seqs]), i32(self.starts))
        w.wal_attn_paged(d, self.cache, *self.args, self.Q, out, ws, scale=scale, max_new=new, max_len=most,
                         stream=stream)
        return out

    def check(self, out, scale=None, present=None):
        scale = self.dim ** -0.5 if scale is None else scale
        got = host(out).reshape(-1, self.group * self.heads, self.dim)
        q = host(self.Q).reshape(got.shape)
        for i, (n, new) in enumerate(self.seqs):
            a, b, rows = self.bounds[i], self.bounds[i] + n, slice(self.starts[i], self.starts[i + 1])
            last = n - new + np.arange(new)
            ref, size, most = A.attend(q[rows], self.k[a:b], self.v[a:b], last, scale,
                                       None if present is None else present[i])
            bound = A.attend_bound(ref, size, most, self.dim, n)
            bad = ~(np.abs(got[rows] - ref) <= bound)
            assert not bad.any(), (i, n, new, np.argwhere(bad)[:3], np.abs(got[rows] - ref).max())


DECODE = [[(1, 1)], [(517, 1)], [(15, 1), (16, 1), (17, 1), (0, 1), (31, 1), (32, 1), (33, 1)],
          [(63, 1), (64, 1), (65, 1), (2, 0), (129, 1), (1000, 1)]]


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("group,heads,dim,page", [(4, 8, 128, 16), (1, 3, 64, 32), (5, 2, 256, 64), (16, 1, 128, 128),
                                                 (17, 2, 64, 16), (64, 1, 128, 256)])
@pytest.mark.parametrize("seqs", range(len(DECODE)))
def test_decode(wal, fmt, group, heads, dim, page, seqs):
    print(f"decode {DECODE[seqs]} group={group} heads={heads} dim={dim} page={page} fmt={fmt}", flush=True)
    p = Paged(wal, DECODE[seqs], group, heads, dim, page, fmt, seed=seqs)
    p.check(p.call())


CHUNKS = [[(7, 7), (64, 64), (100, 3), (1, 1), (0, 0), (65, 65), (3, 5), (0, 2)],    # rows before the first token
          [(130, 130)], [(700, 257), (258, 1), (301, 301), (129, 2)], [(1025, 33)], [(40, 16), (9, 9), (500, 5)]]


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("group,heads,dim,page", [(4, 4, 128, 16), (1, 2, 64, 64), (3, 2, 256, 32), (8, 1, 128, 128),
                                                 (5, 1, 64, 256)])
@pytest.mark.parametrize("seqs", range(len(CHUNKS)))
def test_chunks(wal, fmt, group, heads, dim, page, seqs):
    print(f"chunks {CHUNKS[seqs]} group={group} heads={heads} dim={dim} page={page} fmt={fmt}", flush=True)
    p = Paged(wal, CHUNKS[seqs], group, heads, dim, page, fmt, seed=50 + seqs, pad=16)
    p.check(p.call())
    if p.out.shape[1] > p.Q.shape[1]:
        assert (p.out[:, p.Q.shape[1]:] == 77.0).all()


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("seqs,group,heads,dim", [([(20011, 1)], 4, 2, 128), ([(20011, 1), (5, 1), (3000, 1)], 8, 1, 64),
                                                 ([(9001, 9)], 4, 2, 128), ([(9001, 70), (130, 1)], 4, 1, 128),
                                                 ([(6000, 1)], 2, 2, 256)])
def test_long_context_is_split(wal, fmt, seqs, group, heads, dim):
    print(f"long {seqs} group={group} heads={heads} dim={dim} fmt={fmt}", flush=True)
    p = Paged(wal, seqs, group, heads, dim, 64, fmt, seed=5)
    a = p.call().clone()
    p.check(a)
    assert torch.equal(a, p.call())            # the joining order does not depend on timing


@pytest.mark.parametrize("seqs", [[(300, 1)], [(300, 40)]])
@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (-0.3, 1.0), (1.0, 3.0), (40.0, 1.0)])
def test_scales(wal, seqs, scale, gain):
    """Equal weights, a negative scale, scores of some hundreds: one key takes all."""
    print(f"scale {scale} gain {gain} {seqs}", flush=True)
    p = Paged(wal, seqs, 4, 2, 64, 16, BF16, seed=7, gain=gain)
    p.check(p.call(scale=scale), scale=scale)


def test_one_workspace_for_calls_of_all_sizes(wal):
    """Calls of changing sizes on one workspace, in every order: each leaves its first bytes zero for the next, whose
    partial results lie elsewhere."""
    cases = [Paged(wal, [(3000, 1), (40, 1), (1100, 1), (0, 1)], 4, 2, 128, 16, BF16, seed=21),
             Paged(wal, [(2500, 2), (2100, 1)], 8, 1, 64, 64, INT8, seed=22),
             Paged(wal, [(9001, 40)], 4, 1, 128, 64, BF16, seed=23), Paged(wal, [(30000, 1)], 4, 2, 128, 64, INT8, seed=24),
             Paged(wal, [(1500 + 7 * i, 1) for i in range(40)], 2, 2, 64, 16, BF16, seed=25)]
    size = max(wal.wal_attn_paged_workspace_size(p.d, p.group * p.heads, len(p.seqs), p.Q.shape[0], p.max_new, p.max_len)
               for p in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device=dev())
    want = [p.call().clone() for p in cases]
    for order in ([0, 1, 2, 3, 4], [4, 0, 3, 1, 2], [2, 2, 4, 4, 1, 0, 3]):
        for i in order:
            assert torch.equal(cases[i].call(ws=ws), want[i]), (order, i)
            assert not ws[:wal.WAL_ATTN_WS_ZERO_BYTES].any()
    for p, w in zip(cases, want):
        p.check(w)


def test_bounds_larger_than_the_sequences(wal):
    for seqs in ([(517, 1), (3, 1)], [(300, 40), (7, 2)]):
        p = Paged(wal, seqs, 4, 2, 128, 16, BF16, seed=8)
        p.tables = np.concatenate([p.tables, np.full((len(seqs), 300), -1)], 1)
        p.check(p.call(slack=(30, 4000)))


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("seqs", [[(200, 1), (40, 1)], [(200, 77), (40, 40)]])
def test_pages_outside_the_cache_are_left_out(wal, fmt, seqs):
    p = Paged(wal, seqs, 4, 2, 128, 16, fmt, seed=9)
    present = [np.ones(n, bool) for n, _ in seqs]
    for i, page, bad in ((0, 0, -1), (0, 5, p.d.n_pages), (0, 12, 2 ** 31 - 1), (1, 0, -2 ** 31), (1, 1, -1), (1, 2, -1)):
        p.tables[i, page] = bad
        present[i][16 * page:16 * page + 16] = False
    p.check(p.call(), present=present)         # the second sequence sees nothing: zeros


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("new", [1, 50])
def test_nan_and_infinity(wal, fmt, new):
    """A NaN among the keys a row sees makes the row NaN; one it does not see does not touch it."""
    n, heads, dim = 120, 2, 128
    p = Paged(wal, [(n, new), (80, new)], 4, heads, dim, 16, fmt, seed=11)
    bad = n - new // 2 - 1                     # seen by the later half of the rows (by the only row)
    K = torch.from_numpy(p.k[bad:bad + 1].reshape(1, -1).astype(np.float32)).to(dev())
    K[0, 5] = float("nan")                     # head 0 only
    V = torch.from_numpy(p.v[bad:bad + 1].reshape(1, -1).astype(np.float32)).to(dev())
    wal.wal_kv_write(p.d, p.cache, p.slots[bad:bad + 1], K, V)
    out = p.call()
    got = out.float().cpu().numpy().reshape(2 * new, 4 * heads, dim)
    sees = n - new + np.arange(new) >= bad
    assert np.isnan(got[:new][sees][:, :4]).all() and np.isfinite(got[:new][~sees]).all()
    assert np.isfinite(got[:new, 4:]).all() and np.isfinite(got[new:]).all()
    # the same of v, in the last token, which only the last row sees
    V[0, 3] = float("inf")
    K[0, 5] = 0.0
    wal.wal_kv_write(p.d, p.cache, p.slots[bad:bad + 1], K, V)
    got = p.call().float().cpu().numpy().reshape(2 * new, 4 * heads, dim)
    assert np.isfinite(got[:new][~sees]).all() and not np.isfinite(got[:new][sees][:, :4, 3]).any()
    assert np.isfinite(got[:new, 4:]).all() and np.isfinite(got[new:]).all()


PROMPTS = [[1], [64, 1, 0, 63, 65, 2], [777, 129, 130, 31], [1500]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("group,heads,dim", [(4, 2, 128), (1, 3, 64), (5, 2, 256), (12, 1, 64)])
@pytest.mark.parametrize("lens", range(len(PROMPTS)))
def test_prompt(wal, causal, group, heads, dim, lens):
    lens = PROMPTS[lens]
    print(f"prompt {lens} group={group} heads={heads} dim={dim} causal={causal}", flush=True)
    rng = np.random.default_rng(sum(lens) + dim)
    starts = np.concatenate([[0], np.cumsum(lens)])
    total, qw, kw = starts[-1], group * heads * dim, heads * dim
    wide = t16(rng.standard_normal((total, qw + 2 * kw + 8)))
    Q, K, V = wide[:, :qw], wide[:, qw:qw + kw], wide[:, qw + kw:qw + 2 * kw]
    out = torch.full((total + 1, qw + 24), 77.0, dtype=torch.bfloat16, device=dev())
    wal.wal_attn_prompt(Q, K, V, i32(starts), out[:total, :qw], dim, max(lens), causal=causal)
    assert (out[total] == 77.0).all() and (out[:, qw:] == 77.0).all()
    got = host(out[:total, :qw]).reshape(total, -1, dim)
    q, k, v = (host(x).reshape(total, -1, dim) for x in (Q, K, V))
    for a, b in zip(starts[:-1], starts[1:]):
        last = np.arange(b - a) if causal else np.full(b - a, b - a - 1)
        ref, size, most = A.attend(q[a:b], k[a:b], v[a:b], last, dim ** -0.5)
        assert (np.abs(got[a:b] - ref) <= A.attend_bound(ref, size, most, dim, b - a)).all()


def test_prompt_equals_chunks_over_the_cache(wal):
    """A prompt at once, and the same tokens through a bf16 cache in uneven chunks and a last single token."""
    n, group, heads, dim, page = 333, 4, 2, 128, 16
    Q, K, V = (torch.randn((n, h * dim), device=dev()).to(torch.bfloat16) for h in (group * heads, heads, heads))
    whole = torch.empty_like(Q)
    wal.wal_attn_prompt(Q, K, V, i32([0, n]), whole, dim, n)
    d = wal.make_kv_desc(21, page, heads, dim, BF16)
    cache = new_cache(wal, d, 0xFF)
    pages = np.random.default_rng(3).permutation(21)
    out, at = torch.empty_like(Q), 0
    for c in (100, 17, 1, 64, 150, 1):
        j = np.arange(at, at + c)
        wal.wal_kv_write(d, cache, i32(pages[j // page] * page + j % page), K[at:at + c], V[at:at + c])
        at += c
        ws = torch.zeros(max(16, wal.wal_attn_paged_workspace_size(d, 8, 1, c, c, at)), dtype=torch.uint8, device=dev())
        wal.wal_attn_paged(d, cache, i32(pages[None]), i32([at]), i32([0, c]), Q[at - c:at], out[at - c:at], ws,
                           max_new=c, max_len=at)
    q, k, v = (host(x).reshape(n, -1, dim) for x in (Q, K, V))
    ref, size, most = A.attend(q, k, v, np.arange(n), dim ** -0.5)
    for got in (whole, out):
        assert (np.abs(host(got).reshape(ref.shape) - ref) <= A.attend_bound(ref, size, most, dim, n)).all()


def test_offsets_past_32_bits(wal):
    """Pages at the end of a cache whose planes are 5 GB each."""
    for fmt, pages in ((BF16, 40000), (INT8, 40000)):
        for seqs in ([(150, 1), (40, 1)], [(150, 30), (40, 40)]):
            p = Paged(wal, seqs, 4, 8, 128, 64, fmt, seed=13, pages=pages)
            p.check(p.call())
            del p
            torch.cuda.empty_cache()


def test_bad_sequence_bounds_stay_inside(wal):
    """starts, lens that lie (past the rows, past max_len, falling): some rows get other values, nothing outside is
    read or written (rows and lengths are cut to what the call was told)."""
    p = Paged(wal, [(100, 4), (60, 4)], 4, 2, 128, 16, BF16, seed=17)
    wide = torch.full((9, 1024), 77.0, dtype=torch.bfloat16, device=dev())
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev())
    for starts, lens in (([0, 4, 900], [100, 60]), ([0, 4, 8], [100, 10 ** 9]), ([0, 8, 4], [100, 60]),
                         ([3, 4, 8], [-5, 60]), ([-2 ** 31, 4, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31])):
        wal.wal_attn_paged(p.d, p.cache, i32(p.tables), i32(lens), i32(starts), p.Q, wide[:8], ws, max_new=4, max_len=100)
        wal.wal_attn_prompt(p.Q, p.Q[:, :256], p.Q[:, 256:512], i32(starts), wide[:8], 128, 4)
    torch.cuda.synchronize()
    assert (wide[8] == 77.0).all()


def test_streams_and_graph_replays(wal):
    """A decode step (write, attention) on another stream, and captured: every replay equals the eager result, with
    eager work and other lengths' calls between them."""
    p = Paged(wal, [(700, 1), (33, 1)], 4, 2, 128, 16, INT8, seed=19)
    want = p.call().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.call(out=torch.zeros_like(want))
    s.synchronize()
    assert torch.equal(got, want)
    d = p.d
    n = wal.wal_attn_paged_workspace_size(d, 8, 2, 2, 1, 700)
    ws, out = torch.zeros(max(n, 16), dtype=torch.uint8, device=dev()), torch.zeros_like(want)
    tables, lens, starts = p.args
    turns, _, m = table(wal, 128, "plain", 1.0)
    K, V, Q = (torch.randn((2, h * 128), device=dev()) for h in (2, 2, 8))
    at = [699, 700 + 32]
    slots, pos, q_out = p.slots[at].contiguous(), i32([699, 32]), torch.zeros_like(want)

    def step():
        wal.wal_kv_write(d, p.cache, slots, K, V, pos=pos, turns=turns, magnitude=m, Q=Q, Q_out=q_out)
        wal.wal_attn_paged(d, p.cache, tables, lens, starts, q_out, out, ws, max_new=1, max_len=700)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(5):
        Q.normal_()
        V.normal_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        seen = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(seen, out), i
