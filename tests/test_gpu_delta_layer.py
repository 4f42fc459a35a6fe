"""The layers with the head norms and with the delta rule on small packed matrices: prompts, chunks and single tokens
through the kept states and the cache, and both layers in turn as blocks of a model.

Tolerances, fixed before the first run.  DeltaLayer, per stage on the layer's own tensors: the convolution within the
oracle's conv_bound; the delta rule within 3e-3 of the float64 recurrence on the convolution's own outputs (relative
2-norm: 1.7e-3 is the rounding of the outputs to bf16, and the oracle's tests hold the elements); the gated norm of the
rounded outputs within 2^-8 + 2^-18 of each element.  States taken in pieces against the whole: 1e-5 of their norm.
AttentionLayer with norms: as its test without, with the normed values' 2^-19 more: the oracle's bound and what the
rounding of q and k to bf16 moves the weights by."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import blocks as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HIDDEN, HEADS = 512, dict(key_heads=2, value_heads=4, key_dim=64, value_dim=64)


@pytest.fixture(scope="module")
def mod():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    from ternary_hybrid_bit_amd import attention, delta
    return attention, delta


@pytest.fixture(scope="module")
def parts(mod):
    return mod[1].packed_delta_layer(5, HIDDEN, **HEADS)


def host(t):
    return t.double().cpu().numpy()


def inputs(n, seed=3):
    return torch.randn((n, HIDDEN), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(torch.bfloat16)


def test_stages_against_the_oracle(mod, parts, monkeypatch):
    """Each operator that prompt() calls, on what it was given."""
    _, delta = mod
    layer, seen = delta.DeltaLayer(*parts, **HEADS, max_seqs=1), {}
    for name in ("wal_conv", "wal_delta", "wal_head_norm"):
        def record(*a, _f=getattr(delta, name), _n=name, **kw):
            before = [t.clone() if torch.is_tensor(t) else t for t in a]
            r = _f(*a, **kw)
            seen[_n] = (before, kw, r.clone())
            return r
        monkeypatch.setattr(delta, name, record)
    lens = [70, 1, 130]
    Y = layer.prompt(inputs(sum(lens)), lens)
    assert Y.shape == (sum(lens), HIDDEN) and torch.isfinite(Y).all()
    (x, w, starts, _), kw, got = seen["wal_conv"]
    starts = host(starts).astype(int)
    ref, _, size = B.conv(host(x), host(w), None, starts, np.zeros((0, 3, x.shape[1])), [-1] * 3, True)
    assert (np.abs(host(got) - ref) <= B.conv_bound(ref, size, 4, True, True)).all()
    (d, q, k, v, a, b, *_), kw, got = seen["wal_delta"]
    alpha, beta = B.gates(host(a), host(b), host(kw["decay"]), host(kw["shift"]))
    heads = lambda t: host(t).reshape(t.shape[0], -1, 64)  # noqa: E731
    ref, *_ = B.delta(heads(q), heads(k), heads(v), alpha, beta, starts, np.zeros((0, 4, 64, 64)), [-1] * 3, 1e-6, 0.125, 0.0)
    assert np.linalg.norm(heads(got) - ref) <= 3e-3 * np.linalg.norm(ref)
    (x, _, w, _), kw, got = seen["wal_head_norm"]
    ref = B.head_norm(heads(x), host(w), 1e-6) * B.silu(heads(kw["gate"]))
    assert (np.abs(heads(got) - ref) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(ref) + 1e-30).all()


def test_prompts_chunks_and_tokens(mod, parts):
    layer = mod[1].DeltaLayer(*parts, **HEADS, max_seqs=3)
    lens = [100, 40, 7]
    X = inputs(sum(lens))
    starts = np.cumsum([0] + lens)
    whole = mod[1].DeltaLayer(*parts, **HEADS, max_seqs=3)
    want = whole.forward(X, [0, 1, 2], lens)
    scored = layer.prompt(X, lens)
    assert not layer.state.any() and not layer.rows.any()
    assert torch.equal(scored, want)
    got, done = torch.full_like(want, float("nan")), [0, 0, 0]
    for step in ([70, 20, 0], [1, 1, 1], [0, 16, 2], [28, 1, 4], [1, 2, 0]):
        seqs = [i for i in (2, 0, 1) if step[i]]
        rows = torch.from_numpy(np.concatenate([np.arange(starts[i] + done[i], starts[i] + done[i] + step[i]) for i in seqs])).cuda()
        got[rows] = layer.forward(X[rows], seqs, [step[i] for i in seqs])
        for i in seqs:
            done[i] += step[i]
    assert done == lens
    assert torch.equal(layer.rows, whole.rows) or (layer.rows - whole.rows).norm() <= 1e-5 * whole.rows.norm()
    assert (layer.state - whole.state).norm() <= 1e-5 * whole.state.norm()
    # outputs: two roundings to bf16 before the o product at other places, each 1.7e-3 of the whole
    assert (got - want).norm() <= 8e-3 * want.norm()
    layer.release(1)
    assert not layer.state[1].any() and not layer.rows[1].any() and layer.state[0].any()
    again = layer.forward(X[100:140], [1], [40])
    assert (again - want[100:140]).norm() <= 8e-3 * want[100:140].norm()


def test_refused_calls_change_nothing(mod, parts):
    layer = mod[1].DeltaLayer(*parts, **HEADS, max_seqs=2)
    X = inputs(6)
    layer.forward(X, [0, 1], [4, 2])
    state, rows = layer.state.clone(), layer.rows.clone()
    for seqs, new in (([0], [5]), ([0, 0], [3, 3]), ([0, 2], [3, 3]), ([-1], [6]), ([0, 1], [7, -1]), ([0, 1], [6]), ([], [])):
        with pytest.raises(ValueError):
            layer.forward(X, seqs, new)
    with pytest.raises(ValueError):
        layer.release(2)
    with pytest.raises(TypeError):
        layer.forward(X.float().half(), [0, 1], [4, 2])
    assert torch.equal(layer.state, state) and torch.equal(layer.rows, rows)


def test_attention_with_head_norms(mod):
    qh, kvh, d = 8, 2, 64
    mats = mod[0].packed_layer(11, HIDDEN, qh, kvh, d)
    g = torch.Generator("cuda").manual_seed(4)
    q_norm, k_norm = (1 + 0.3 * torch.randn(d, device="cuda", generator=g) for _ in range(2))
    layer = mod[0].AttentionLayer(*mats, head_dim=d, n_pages=20, max_seqs=2, page_size=16, q_norm=q_norm, k_norm=k_norm)
    lens = [70, 33]
    X = inputs(sum(lens), 6)
    Q, K, V = (layer._product(m, X) for m in layer.mats[:3])
    f, m = A.rope_freqs(d, 1e6)
    heads = lambda t: host(t).reshape(t.shape[0], -1, d)  # noqa: E731
    v = heads(V.to(torch.bfloat16))
    ref, bound, at = [], [], 0
    for n in lens:
        pos, s = np.arange(n), slice(at, at + n)
        qr = A.rope(B.head_norm(heads(Q)[s], host(q_norm), 1e-6), pos, f, m)[0]
        kr = A.rope(B.head_norm(heads(K)[s], host(k_norm), 1e-6), pos, f, m)[0]
        o, size, most = A.attend(qr, kr, v[s], pos, d ** -0.5)
        ref.append(o)
        bound.append(A.attend_bound(o, size, most, d, n) + 2 * np.expm1(2.1 * (2.0 ** -8 + 2.0 ** -18) * most)[..., None] * size)
        at += n
    ref, bound = (np.concatenate(t).reshape(X.shape[0], -1) for t in (ref, bound))
    first = layer.attend(Q[:69], K[:69], V[:69], [0], [69])
    rest = layer.attend(Q[69:], K[69:], V[69:], [0, 1], [1, 33])
    got = np.concatenate([host(first), host(rest)])
    assert (np.abs(got - ref) <= bound).all()
    # prompt() makes the same numbers by wal_head_norm (its o product is on attend()'s own rounded outputs here)
    want = layer._product(layer.mats[3], torch.cat([first, rest]))
    assert (layer.prompt(X, lens) - want).norm() <= 8e-3 * want.norm()
    plain = mod[0].AttentionLayer(*mats, head_dim=d, n_pages=20, max_seqs=2, page_size=16)
    assert not torch.equal(plain.prompt(X, lens), layer.prompt(X, lens))


def test_blocks_in_turn(mod, parts):
    """Three delta-rule blocks and one of attention with head norms, prompts and then tokens, against whole prompts."""
    qh, kvh, d = 8, 2, 64
    w = torch.ones(d, device="cuda")
    delta = [mod[1].DeltaLayer(*mod[1].packed_delta_layer(20 + i, HIDDEN, **HEADS), **HEADS, max_seqs=2) for i in range(3)]
    attn = mod[0].AttentionLayer(*mod[0].packed_layer(30, HIDDEN, qh, kvh, d), head_dim=d, n_pages=12, max_seqs=2, page_size=16,
                                 q_norm=w, k_norm=w)

    def model(X, call):
        x = X
        for block in (*delta, attn):
            y = call(block, x)
            x = (x.float() + y / y.norm(dim=1, keepdim=True) * 4).to(torch.bfloat16)
        return x

    X = inputs(100, 8)
    whole = model(X, lambda b, x: b.prompt(x, [64, 36]))
    first = model(torch.cat([X[:62], X[64:99]]), lambda b, x: b.forward(x, [1, 0], [62, 35]))
    tokens = [model(torch.cat([X[62 + i:63 + i], X[99:100]] if i else [X[62:63]]), lambda b, x: b.forward(x, [1, 0][:1 + i], [1] * (1 + i)))
              for i in range(2)]
    got = torch.cat([first[:62], tokens[0], tokens[1][:1], first[62:], tokens[1][1:]]).float()
    assert torch.isfinite(got).all()
    # four blocks of roundings to bf16 in other places: each 2^-8 of a row at most
    assert (got - whole.float()).norm() <= 4 * 2.0 ** -8 * whole.float().norm()
