"""GPU tests of wal_head_norm and of the norms in wal_kv_write against float64 (oracle/blocks.py, oracle/attention.py).

Tolerances, fixed before the first run:
* normed values: 2^-19 of the value.  The sum of dim squares takes up to 16 fused steps, 5 exchanges, a scaling and eps:
  at most 23 roundings of 2^-24, half of which reach the root; the root, the quotient, the products with the weight and
  the element 4 more, of up to 2^-23: below 20 * 2^-24.
* silu(gate): its exponential (2^-22), sum, quotient and two products: 2^-20 of the value more, and where the
  exponential overflows 2^-100 in all (88 exp(-88) is 5e-37);
* the rotation: 2^-21 (|a| + |b|) of normed values as for wal_rope, whose own errors come with them (2^-19 (|a| + |b|));
* bf16 output: 2^-8 of the value more; int8 rows: half a step of the row's scale (which is max / 127, fp32).
"""
import numpy as np
import pytest

from oracle import attention as A
from oracle import blocks as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f": torch.float32, "b": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module")
def wal():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import ternary_hybrid_bit_amd as w
    return w


def host(t):
    return t.double().cpu().numpy()


def padded(x, pad, dtype):
    """x on the GPU inside rows that are pad wider, NaN around it."""
    t = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :x.shape[1]] = torch.from_numpy(np.asarray(x, np.float32)).cuda().to(dtype)
    return t[:, :x.shape[1]]


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


def vector(rng, dim, t):
    return torch.from_numpy((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)).cuda().to(TYPES[t])


def turns_of(wal, rot):
    return torch.from_numpy(wal.wal_rope_freqs(wal.make_rope_desc(rot, 1e6))[0]).cuda()


def rotated_oracle(y, pos, rot, interleaved):
    f, m = A.rope_freqs(rot, 1e6)
    return A.rope(y, pos, f, m, interleaved)


@pytest.mark.parametrize("n,heads,dim,tin,tw,tout,pad,then", [
    (1, 48, 128, "b", "b", "b", 0, "gate f"), (1, 1, 16, "f", "f", "f", 0, ""), (3, 5, 80, "f", "b", "f", 8, "gate b"),
    (2, 3, 48, "b", "f", "f", 16, ""), (37, 40, 128, "f", "b", "b", 0, "rot 128"), (130, 3, 192, "b", "f", "b", 64, "rot 64 i"),
    (5, 2, 512, "b", "b", "f", 0, "rot 512 i"), (2111, 13, 256, "f", "f", "b", 64, "rot 64"), (1000, 7, 96, "f", "b", "f", 0, "rot 96"),
    (4097, 10, 64, "b", "f", "f", 0, "gate b"), (3001, 48, 128, "b", "b", "b", 128, "gate f"), (17, 31, 336, "f", "f", "b", 0, "gate f"),
])
def test_head_norm(wal, n, heads, dim, tin, tw, tout, pad, then):
    print(f"norm n={n} heads={heads} dim={dim} {tin}{tw}->{tout} pad={pad} {then}", flush=True)
    rng = np.random.default_rng(n + dim)
    X = padded(rng.standard_normal((n, heads * dim)) * np.exp(rng.standard_normal(heads * dim)), pad, TYPES[tin])
    w = vector(rng, dim, tw)
    whole = torch.full((n, heads * dim + pad), float("nan"), dtype=TYPES[tout], device="cuda")
    out, kw = whole[:, :heads * dim], {}
    kind = then.split()
    if kind and kind[0] == "gate":
        kw["gate"] = padded(3 * rng.standard_normal((n, heads * dim)), pad, TYPES[kind[1]])
        kw["gate"][0, 0], kw["gate"][n - 1, 1] = -300.0, 300.0
    if kind and kind[0] == "rot":
        pos, rot = rng.integers(0, 1 << 16, n), int(kind[1])
        kw.update(pos=i32(pos), turns=turns_of(wal, rot), layout=int(len(kind) > 2))
    assert wal.wal_head_norm(X, out, w, dim, eps=EPS, **kw) is out
    torch.cuda.synchronize()
    ref = B.head_norm(host(X).reshape(n, heads, dim), host(w), EPS)
    bound = 2.0 ** -19 * np.abs(ref)
    if kind and kind[0] == "rot":
        ref, size = rotated_oracle(ref, pos, rot, len(kind) > 2)
        # positions below 2^16: the angle's own rounding in float64 is nothing; copied elements keep the norm's bound
        bound = np.where(size > 0, (2.0 ** -21 + 2.0 ** -19) * size, bound)
    if kind and kind[0] == "gate":
        ref = ref * B.silu(host(kw["gate"]).reshape(ref.shape))
        bound = (2.0 ** -19 + 2.0 ** -20) * np.abs(ref) + 2.0 ** -100
    if tout == "b":
        bound = bound + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(host(out).reshape(ref.shape) - ref) <= bound).all()
    if pad:
        assert torch.isnan(whole[:, heads * dim:]).all()


@pytest.mark.parametrize("then", ["", "gate", "rot"])
@pytest.mark.parametrize("t", ["f", "b"])
def test_in_place_and_repeated(wal, t, then):
    X = torch.randn((301, 6 * 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(TYPES[t])
    w, kw = vector(np.random.default_rng(1), 128, "f"), {}
    if then == "gate":
        kw["gate"] = X.flip(0).contiguous()
    if then == "rot":
        kw.update(pos=i32(np.arange(301)), turns=turns_of(wal, 64))
    out = [wal.wal_head_norm(X, torch.empty_like(X), w, 128, **kw) for _ in range(2)]
    wal.wal_head_norm(X, X, w, 128, **kw)
    assert torch.equal(X, out[0]) and torch.equal(out[0], out[1])


@pytest.mark.parametrize("t", ["f", "b"])
def test_sizes_of_values(wal, t):
    """Zeros, values whose squares pass or fall below fp32's range, infinities and NaN: each head for itself."""
    dim, heads = 80, 7
    x = np.random.default_rng(2).standard_normal((1, heads, dim))
    x[0, 0], x[0, 1], x[0, 2] = 0.0, x[0, 1] * 1e30, x[0, 2] * 1e-30
    x[0, 3, 5], x[0, 4, 6] = np.inf, np.nan
    x[0, 5] = 3.3e38 * np.sign(x[0, 5])
    X = padded(x.reshape(1, -1), 0, TYPES[t])
    w, out = torch.ones(dim, device="cuda"), torch.empty((1, heads * dim), device="cuda")
    wal.wal_head_norm(X, out, w, dim, eps=EPS)
    got, xs = host(out).reshape(heads, dim), host(X).reshape(heads, dim)
    for h in (0, 1, 2, 5, 6):
        ref = B.head_norm(xs[None, None, h], np.ones(dim), EPS)[0, 0]
        assert (np.abs(got[h] - ref) <= 2.0 ** -19 * np.abs(ref) + 1e-44).all(), h
    assert np.isnan(got[3, 5]) and (np.delete(got[3], 5) == 0).all()
    assert np.isnan(got[4]).all()


def test_small_and_large_eps(wal):
    x = np.random.default_rng(3).standard_normal((4, 128))
    X, w, out = padded(x, 0, torch.float32), torch.ones(64, device="cuda"), torch.empty((4, 128), device="cuda")
    for eps in (1e-37, 1e-3, 50.0, 1e30):
        wal.wal_head_norm(X, out, w, 64, eps=eps)
        ref = B.head_norm(host(X).reshape(4, 2, 64), np.ones(64), float(np.float32(eps)))
        assert (np.abs(host(out).reshape(ref.shape) - ref) <= 2.0 ** -19 * np.abs(ref)).all(), eps


# ---- into the cache -----------------------------------------------------------

@pytest.mark.parametrize("n,qh,kvh,dim,rot,layout,tin,tw,fmt,page", [
    (1, 32, 8, 128, 128, 0, "f", "b", 0, 16), (37, 32, 8, 128, 128, 0, "f", "f", 1, 16), (301, 6, 2, 256, 64, 1, "b", "b", 0, 64),
    (70, 5, 5, 64, 32, 0, "b", "f", 1, 32), (2500, 8, 4, 64, 64, 1, "f", "b", 1, 128),
])
def test_normed_write(wal, n, qh, kvh, dim, rot, layout, tin, tw, fmt, page):
    print(f"write n={n} {qh}/{kvh} heads of {dim} rot={rot} {layout} {tin}{tw} fmt={fmt} page={page}", flush=True)
    rng = np.random.default_rng(n)
    d = wal.make_kv_desc(-(-n // page) + 2, page, kvh, dim, fmt)
    cache = torch.zeros(wal.wal_kv_size(d).total_bytes, dtype=torch.uint8, device="cuda")
    slots = rng.permutation(d.n_pages * page)[:n]
    slots[n // 2] = d.n_pages * page if n > 2 else slots[n // 2]       # one token that is dropped
    Q, K, V = (padded(rng.standard_normal((n, h * dim)) * np.exp(rng.standard_normal(h * dim)), 8, TYPES[tin]) for h in (qh, kvh, kvh))
    q_norm, k_norm = vector(rng, dim, tw), vector(rng, dim, tw)
    pos, turns = rng.integers(0, 1 << 16, n), turns_of(wal, rot)
    q_out = torch.full((n, qh * dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    wal.wal_kv_write(d, cache, i32(slots), K, V, pos=i32(pos), turns=turns, layout=layout, Q=Q, Q_out=q_out, q_norm=q_norm,
                     k_norm=k_norm, eps=EPS)
    k, v = (torch.full((n, kvh * dim), float("nan"), device="cuda") for _ in range(2))
    wal.wal_kv_read(d, cache, i32(slots), k, v)
    heads = lambda t: host(t).reshape(n, -1, dim)  # noqa: E731

    def turned(x, w):
        y, size = rotated_oracle(B.head_norm(heads(x), host(w), EPS), pos, rot, layout == 1)
        return y, np.where(size > 0, (2.0 ** -21 + 2.0 ** -19) * size, 2.0 ** -19 * np.abs(y))

    ref, err = turned(Q, q_norm)
    assert (np.abs(heads(q_out) - ref) <= err + 2.0 ** -8 * np.abs(ref)).all()
    ref, err = turned(K, k_norm)
    live = slots < d.n_pages * page
    ref, err = ref[live], err[live]
    if fmt == 0:
        assert (np.abs(heads(k)[live] - ref) <= err + 2.0 ** -8 * np.abs(ref)).all()
        assert np.array_equal(heads(v)[live], host(V.to(torch.bfloat16)).reshape(n, -1, dim)[live])
    else:
        top = np.abs(ref).max(-1, keepdims=True)
        most = err.max(-1, keepdims=True)
        assert (np.abs(heads(k)[live] - ref) <= 0.5 * (top + most) / 127 * (1 + 2.0 ** -20) + most + 2.0 ** -22 * top).all()
        codes, scale = A.int8_rows(heads(V))
        assert np.array_equal(heads(v)[live], (codes * scale[..., None]).astype(np.float32).astype(np.float64)[live])
    assert (heads(k)[~live] == 0).all()


def test_write_norms_one_side_and_equals_two_calls(wal):
    """k alone, q alone, both: the same bits as wal_head_norm in fp32 followed by the write (fp32 rows are not rounded)."""
    n, qh, kvh, dim = 65, 4, 2, 128
    g = torch.Generator("cuda").manual_seed(5)
    Q, K, V = (torch.randn((n, h * dim), device="cuda", generator=g) for h in (qh, kvh, kvh))
    w = [vector(np.random.default_rng(i), dim, "f") for i in (1, 2)]
    d = wal.make_kv_desc(5, 16, kvh, dim, 0)
    slots, pos, turns = i32(np.arange(n)), i32(np.arange(n)), turns_of(wal, 64)

    def write(Q, K, **kw):
        cache, q = torch.zeros(wal.wal_kv_size(d).total_bytes, dtype=torch.uint8, device="cuda"), torch.empty(Q.shape, dtype=torch.bfloat16, device="cuda")
        wal.wal_kv_write(d, cache, slots, K, V, pos=pos, turns=turns, Q=Q, Q_out=q, **kw)
        return cache, q

    normed = [wal.wal_head_norm(x, torch.empty_like(x), v, dim) for x, v in ((Q, w[0]), (K, w[1]))]
    for kw, a, b in ((dict(q_norm=w[0], k_norm=w[1]), normed[0], normed[1]), (dict(k_norm=w[1]), Q, normed[1]), (dict(q_norm=w[0]), normed[0], K)):
        for x, y in zip(write(Q, K, **kw), write(a, b)):
            assert torch.equal(x, y)


def test_under_graph_and_on_another_stream(wal):
    X = torch.randn((7, 512), device="cuda")
    w, gate, out = torch.ones(64, device="cuda"), torch.randn((7, 512), device="cuda"), torch.empty((7, 512), device="cuda")
    want = wal.wal_head_norm(X, torch.empty_like(X), w, 64, gate=gate).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        wal.wal_head_norm(X, out, w, 64, gate=gate)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wal.wal_head_norm(X, out, w, 64, gate=gate)
    for i in range(3):
        X.copy_(torch.randn((7, 512), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wal.wal_head_norm(X, torch.empty_like(X), w, 64, gate=gate))
