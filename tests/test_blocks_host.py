"""The oracle of the head norms, the convolution and the delta rule (oracle/blocks.py) against cases worked by hand
and against other ways to the same numbers; what the library and the binding refuse, without a GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import ternary_hybrid_bit_amd as wal
from oracle import blocks as B

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
ARG, SHAPE, BUFFER, ALIGN = -1, -2, -5, -6


# ---- the oracle ---------------------------------------------------------------

def test_head_norm_by_hand():
    # mean square (9 + 16 + 0 + 0) / 4 = 6.25, root 2.5
    y = B.head_norm([[[3.0, -4.0, 0.0, 0.0]]], [1.0, 2.0, 1.0, 1.0], 0.0)
    assert np.allclose(y, [[[1.2, -3.2, 0.0, 0.0]]], rtol=1e-15)
    assert np.allclose(B.head_norm(np.zeros((1, 1, 4)), np.ones(4), 1e-6), 0.0)


def test_conv_is_a_convolution_and_can_be_cut_anywhere():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((20, 8)), rng.standard_normal((8, 4))
    zero = np.zeros((1, 3, 8))
    out, last, _ = B.conv(x, w, None, [0, 20], zero, [0], False)
    for c in range(8):
        assert np.allclose(out[:, c], np.convolve(x[:, c], w[c, ::-1])[:20])
    assert np.array_equal(last[0], x[-3:])
    for cut in (1, 2, 7, 19):
        a, state, _ = B.conv(x[:cut], w, None, [0, cut], zero, [0], False)
        b, state, _ = B.conv(x[cut:], w, None, [0, 20 - cut], state, [0], False)
        assert np.allclose(np.concatenate([a, b]), out) and np.array_equal(state, last)


def test_delta_rule_stores_replaces_and_forgets():
    # one head, keys along the axes: a state is a table of rows
    k = np.eye(4)[[0, 1, 0]][:, None, :]
    v = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])[:, None, :]
    one = np.ones((3, 1))
    out, state, _, _ = B.delta(k, k, v, one, one, [0, 3], np.zeros((1, 1, 4, 2)), [0], 0.0, 1.0, 0.0)
    assert np.array_equal(out[:, 0], v[:, 0])                                   # what was stored is read back
    assert np.array_equal(state[0, 0], [[5, 6], [3, 4], [0, 0], [0, 0]])        # the first row replaced, not added to
    half = np.full((3, 1), 0.5)
    _, state, _, _ = B.delta(k, k, v, half, one, [0, 3], np.zeros((1, 1, 4, 2)), [0], 0.0, 1.0, 0.0)
    assert np.array_equal(state[0, 0], [[5, 6], [1.5, 2], [0, 0], [0, 0]])      # halved once after it was written
    _, state, _, _ = B.delta(k, k, v, one, half, [0, 3], np.zeros((1, 1, 4, 2)), [0], 0.0, 1.0, 0.0)
    assert np.array_equal(state[0, 0], [[2.75, 3.5], [1.5, 2], [0, 0], [0, 0]])  # half of the way from (0.5, 1) to (5, 6)


def test_delta_rule_equals_its_product_form():
    """S_t = S_{t-1} alpha (1 - beta k k^T) + beta v k^T, written as matrices, in any cutting of the sequence."""
    rng = np.random.default_rng(2)
    n, d, e = 12, 6, 5
    q, k, v = rng.standard_normal((n, 1, d)), rng.standard_normal((n, 1, d)), rng.standard_normal((n, 1, e))
    alpha, beta = rng.uniform(0.5, 1, (n, 1)), rng.uniform(0, 1, (n, 1))
    start = rng.standard_normal((1, 1, d, e))
    out, state, _, _ = B.delta(q, k, v, alpha, beta, [0, n], start, [0], 1e-6, 0.3, 0.0)
    unit = lambda x: x / math.sqrt(x @ x + 1e-6)  # noqa: E731
    m = start[0, 0].T
    for t in range(n):
        kt = unit(k[t, 0])
        m = m @ (alpha[t, 0] * (np.eye(d) - beta[t, 0] * np.outer(kt, kt))) + beta[t, 0] * np.outer(v[t, 0], kt)
        assert np.allclose(out[t, 0], 0.3 * m @ unit(q[t, 0]))
    assert np.allclose(state[0, 0], m.T)
    a = B.delta(q[:5], k[:5], v[:5], alpha[:5], beta[:5], [0, 5], start, [0], 1e-6, 0.3, 0.0)
    b = B.delta(q[5:], k[5:], v[5:], alpha[5:], beta[5:], [0, n - 5], a[1], [0], 1e-6, 0.3, 0.0)
    assert np.allclose(np.concatenate([a[0], b[0]]), out) and np.allclose(b[1], state)


def test_gates():
    alpha, beta = B.gates([[0.0]], [[0.0]], [2.0], [0.0])
    assert np.allclose(alpha, 0.25) and np.allclose(beta, 0.5)       # exp(-2 ln 2)
    alpha, beta = B.gates([[-1.0, 0.5]], [[0.3, 1.5]], None, None)
    assert np.allclose(alpha, [[math.exp(-1), 1.0]]) and np.allclose(beta, [[0.3, 1.5]])


# ---- refusals of the library ----------------------------------------------------
# Host memory stands for device memory: every call below is refused before any launch, or has nothing to do.

def at(n=1 << 16, align=256):
    raw = np.zeros(n + align, np.uint8)
    off = -raw.ctypes.data % align
    return raw, raw.ctypes.data + off


class Norm:
    def __init__(self):
        self.keep = [at() for _ in range(6)]
        x, w, g, out, pos, turns = (p for _, p in self.keep)
        self.r = wal.wal_rotary(turns, pos, 32, 0, 1.0)
        self.args = dict(x=x, xd=1, n=2, heads=2, dim=64, ldx=128, w=w, wd=0, eps=1e-6, r=None, g=None, gd=0, ldg=128,
                         out=out, od=1, ldo=128)
        self.gate = g

    def call(self, **kw):
        a = dict(self.args, **kw)
        return wal._lib.wal_head_norm(a["x"], a["xd"], a["n"], a["heads"], a["dim"], a["ldx"], a["w"], a["wd"], a["eps"],
                                      a["r"], a["g"], a["gd"], a["ldg"], a["out"], a["od"], a["ldo"], None)


def test_head_norm_refusals():
    c = Norm()
    x, w, out, g = c.args["x"], c.args["w"], c.args["out"], c.gate
    r = ctypes.byref(c.r)
    assert c.call(n=0) == 0 and c.call(n=0, r=r) == 0 and c.call(n=0, g=g, gd=1) == 0
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(xd=2), dict(od=16), dict(wd=-1), dict(g=g, gd=3),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(eps=1e-39), dict(r=r, g=g),
               dict(ldx=64), dict(ldo=64), dict(g=g, ldg=64), dict(out=x + 16), dict(out=w, n=1), dict(g=out),
               dict(out=x, ldo=256), dict(out=x, od=0)):
        assert c.call(**kw) == ARG, kw
    for kw in (dict(heads=0), dict(dim=0), dict(dim=72), dict(dim=528, ldx=2048, ldo=2048), dict(n=(1 << 30) + 1),
               dict(heads=65536)):
        assert c.call(**kw) == SHAPE, kw
    for kw in (dict(x=x + 2), dict(out=out + 8), dict(g=g + 4), dict(ldx=132), dict(w=w + 2), dict(w=w + 1, wd=1)):
        assert c.call(**kw) == ALIGN, kw
    c.r.rot_dim = 80
    assert c.call(r=r) == SHAPE


def test_normed_write_refusals():
    d = wal.make_kv_desc(2, 16, 2, 64)
    keep = [at() for _ in range(9)]
    cache, slots, k, v, q, qo, pos, turns, w = (p for _, p in keep)
    r = wal.wal_rotary(turns, pos, 32, 0, 1.0)

    def call(n=0, norms=wal.wal_norms(w, w, 0, 1e-6), q=q, qo=qo):
        return wal._lib.wal_kv_write_normed(ctypes.byref(d), cache, slots, n, k, 128, v, 128, 1,
                                            None if norms is None else ctypes.byref(norms), ctypes.byref(r), q, 2, 128,
                                            qo, 128, None)
    assert call() == 0 and call(norms=wal.wal_norms(None, w, 1, 1e-6), q=None, qo=None) == 0
    for kw in (dict(norms=None), dict(norms=wal.wal_norms(w, w, 2, 1e-6)), dict(norms=wal.wal_norms(w, w, 0, 0.0)),
               dict(norms=wal.wal_norms(w, w, 0, math.nan)), dict(q=None, qo=None),
               dict(n=1, norms=wal.wal_norms(qo, w, 0, 1e-6)), dict(n=1, norms=wal.wal_norms(w, cache, 0, 1e-6))):
        assert call(**kw) == ARG, kw
    assert call(norms=wal.wal_norms(w + 2, w, 0, 1e-6)) == ALIGN and call(norms=wal.wal_norms(w, w + 1, 1, 1e-6)) == ALIGN


def test_conv_refusals():
    keep = [at() for _ in range(7)]
    x, w, b, starts, state, slots, out = (p for _, p in keep)

    def call(**kw):
        a = dict(dict(x=x, xd=1, n=2, c=64, ldx=64, w=w, wd=0, taps=4, b=b, starts=starts, seqs=1, state=state,
                      slots=slots, n_slots=2, out=out, od=1, ldo=64), **kw)
        return wal._lib.wal_conv(a["x"], a["xd"], a["n"], a["c"], a["ldx"], a["w"], a["wd"], a["taps"], a["b"], 1,
                                 a["starts"], a["seqs"], a["state"], a["slots"], a["n_slots"], a["out"], a["od"],
                                 a["ldo"], None)
    assert call(n=0) == 0 and call(seqs=0) == 0 and call(n=0, state=None, slots=None, b=None) == 0
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(starts=None), dict(state=None), dict(slots=None),
               dict(xd=2), dict(wd=2), dict(od=-1), dict(ldx=56), dict(ldo=56), dict(out=x), dict(out=x + 16),
               dict(out=state), dict(state=x), dict(out=w), dict(out=b), dict(state=w), dict(state=starts), dict(out=slots)):
        assert call(**kw) == ARG, kw
    for kw in (dict(c=0), dict(c=60, ldx=64), dict(taps=1), dict(taps=5), dict(n=(1 << 24) + 1), dict(seqs=(1 << 24) + 1),
               dict(n_slots=(1 << 24) + 1), dict(c=(1 << 24) + 8, ldx=(1 << 25), ldo=(1 << 25))):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=x + 8), dict(out=out + 2), dict(w=w + 4), dict(b=b + 2), dict(state=state + 8), dict(starts=starts + 1),
               dict(slots=slots + 2), dict(ldx=68), dict(ldo=65)):
        assert call(**kw) == ALIGN, kw


def delta_call():
    keep = [at(1 << 18) for _ in range(12)]
    q, k, v, a, b, de, sh, starts, state, slots, out, ws = (p for _, p in keep)

    def call(desc=(2, 4, 64, 32, 1e-6, 0.125), **kw):
        x = dict(dict(q=q, ldq=128, k=k, ldk=128, v=v, ldv=128, a=a, lda=4, b=b, ldb=4, de=de, sh=sh, starts=starts,
                      seqs=1, n=2, new=2, state=state, slots=slots, n_slots=2, out=out, ldo=128, ws=ws, wsb=1 << 17), **kw)
        d = None if desc is None else ctypes.byref(wal.wal_delta_desc(*desc))
        return wal._lib.wal_delta(d, x["q"], x["ldq"], x["k"], x["ldk"], x["v"], x["ldv"], x["a"], x["lda"], x["b"],
                                  x["ldb"], x["de"], x["sh"], x["starts"], x["seqs"], x["n"], x["new"], x["state"],
                                  x["slots"], x["n_slots"], x["out"], x["ldo"], x["ws"], x["wsb"], None)
    call.keep, call.at = keep, dict(q=q, k=k, v=v, a=a, b=b, de=de, sh=sh, starts=starts, state=state, slots=slots,
                                    out=out, ws=ws)
    return call


def test_delta_refusals():
    call = delta_call()
    p = call.at
    assert call(n=0) == 0 and call(seqs=0) == 0 and call(new=0) == 0
    assert call(n=0, state=None, slots=None, de=None, sh=None) == 0
    for kw in (dict(desc=None), dict(q=None), dict(k=None), dict(v=None), dict(a=None), dict(b=None), dict(out=None),
               dict(starts=None), dict(state=None), dict(slots=None), dict(de=None), dict(sh=None), dict(ldq=64),
               dict(ldv=64), dict(ldo=64), dict(lda=3), dict(ldb=3), dict(out=p["q"]), dict(out=p["v"]),
               dict(out=p["state"]), dict(state=p["k"]), dict(state=p["b"]), dict(out=p["a"]), dict(out=p["sh"]),
               dict(state=p["slots"]), dict(desc=(2, 4, 64, 32, -1.0, 1.0)), dict(desc=(2, 4, 64, 32, math.nan, 1.0)),
               dict(desc=(2, 4, 64, 32, 1e-40, 1.0)), dict(desc=(2, 4, 64, 32, 0.0, math.inf))):
        assert call(**kw) == ARG, kw
    for kw in (dict(desc=(0, 4, 64, 32, 0, 1)), dict(desc=(3, 4, 64, 32, 0, 1)), dict(desc=(2, 0, 64, 32, 0, 1)),
               dict(desc=(2, 4, 96, 32, 0, 1)), dict(desc=(2, 4, 64, 40, 0, 1)), dict(desc=(2, 4, 64, 288, 0, 1)),
               dict(desc=(1, 1025, 64, 32, 0, 1)), dict(n=(1 << 24) + 1), dict(seqs=(1 << 24) + 1),
               dict(new=(1 << 24) + 1), dict(n_slots=(1 << 24) + 1), dict(ldq=(1 << 24) + 8), dict(ldk=(1 << 24) + 8),
               dict(ldv=(1 << 24) + 8), dict(ldo=(1 << 24) + 8)):
        assert call(**kw) == SHAPE, kw
    for name in ("q", "k", "v", "out", "state"):
        assert call(**{name: p[name] + 8}) == ALIGN, name
    for name in ("a", "b", "de", "sh", "starts", "slots"):
        assert call(**{name: p[name] + 2}) == ALIGN, name
    for kw in (dict(ldq=132), dict(ldk=129), dict(ldv=130), dict(ldo=132)):
        assert call(**kw) == ALIGN, kw


# ---- refusals of the binding -----------------------------------------------------

def meta(*shape, dt=BF, stride=None):
    t = torch.empty(shape, dtype=dt, device="meta")
    return t if stride is None else torch.empty_strided(shape, stride, dtype=dt, device="meta")


def test_binding_head_norm():
    x, w = meta(3, 256), meta(64, dt=F32)
    for bad, err in ((lambda: wal.wal_head_norm(x, x, w, 48), ValueError), (lambda: wal.wal_head_norm(x, x, meta(128), 64), ValueError),
                     (lambda: wal.wal_head_norm(x, x, meta(64, dt=torch.float16), 64), TypeError),
                     (lambda: wal.wal_head_norm(x, x, [1.0] * 64, 64), TypeError),
                     (lambda: wal.wal_head_norm(x, x, meta(64, stride=(2,)), 64), ValueError),
                     (lambda: wal.wal_head_norm(x, meta(2, 256), w, 64), ValueError),
                     (lambda: wal.wal_head_norm(x, meta(3, 192), w, 64), ValueError),
                     (lambda: wal.wal_head_norm(x, x, w, 64, gate=meta(3, 192)), ValueError),
                     (lambda: wal.wal_head_norm(x, x, w, 64, gate=meta(3, 256, dt=I32)), TypeError),
                     (lambda: wal.wal_head_norm(x, x, w, 64, pos=meta(3, dt=I32)), ValueError),
                     (lambda: wal.wal_head_norm(x, x, w, 64, pos=meta(3, dt=I32), turns=meta(32, dt=I64), gate=x), ValueError),
                     (lambda: wal.wal_head_norm(x, x, w, 64, pos=meta(2, dt=I32), turns=meta(32, dt=I64)), ValueError),
                     (lambda: wal.wal_head_norm(meta(2, 256, stride=((1 << 32) + 256, 1)), x, w, 64), ValueError)):
        with pytest.raises(err):
            bad()
    with pytest.raises(ValueError, match="GPU"):
        wal.wal_head_norm(x, x, w, 64)


def test_binding_normed_write():
    d = wal.make_kv_desc(1, 16, 4, 64)
    cache, slots, x = meta(wal.wal_kv_size(d).total_bytes, dt=torch.uint8), meta(2, dt=I32), meta(2, 256)
    pos, turns, w = meta(2, dt=I32), meta(32, dt=I64), meta(64, dt=F32)
    go = lambda **kw: wal.wal_kv_write(d, cache, slots, x, x, **kw)  # noqa: E731
    for kw, err in ((dict(k_norm=meta(128, dt=F32)), ValueError), (dict(q_norm=w), ValueError),
                    (dict(k_norm=w, q_norm=meta(64), pos=pos, turns=turns, Q=x, Q_out=x), TypeError),
                    (dict(k_norm=meta(64, dt=torch.float64)), TypeError)):
        with pytest.raises(err):
            go(**kw)
    with pytest.raises(ValueError, match="GPU"):
        go(k_norm=w, q_norm=w, pos=pos, turns=turns, Q=x, Q_out=x)


def test_binding_conv():
    x, w, starts, out = meta(3, 64, dt=F32), meta(64, 4), meta(3, dt=I32), meta(3, 64)
    state, slots = meta(5, 3, 64, dt=F32), meta(2, dt=I32)
    go = lambda **kw: wal.wal_conv(**dict(dict(X=x, weight=w, starts=starts, out=out, state=state, slots=slots), **kw))  # noqa: E731
    for kw, err in ((dict(state=None), ValueError), (dict(slots=None), ValueError), (dict(weight=meta(32, 4)), ValueError),
                    (dict(weight=meta(64, 4, stride=(8, 1))), ValueError), (dict(state=meta(5, 3, 64)), TypeError),
                    (dict(state=meta(5, 2, 64, dt=F32)), ValueError), (dict(state=meta(5, 192, dt=F32)), ValueError),
                    (dict(state=meta(5, 3, 64, dt=F32, stride=(256, 64, 1))), ValueError), (dict(slots=meta(1, dt=I32)), ValueError),
                    (dict(slots=meta(2, dt=I64)), TypeError), (dict(bias=meta(64, dt=F32)), TypeError),
                    (dict(bias=meta(60)), ValueError), (dict(out=meta(2, 64)), ValueError), (dict(out=meta(3, 56)), ValueError),
                    (dict(starts=meta(0, dt=I32)), ValueError), (dict(starts=meta(3, dt=I64)), TypeError),
                    (dict(out=meta(3, 64, dt=torch.float16)), TypeError)):
        with pytest.raises(err):
            go(**kw)
    with pytest.raises(ValueError, match="GPU"):
        go()


def test_binding_delta():
    d = wal.make_delta_desc(2, 4, 64, 32)
    assert d.scale == pytest.approx(0.125) and wal.make_delta_desc(2, 4, 64, 32, scale=0.5).scale == 0.5
    q, v, g, starts, w = meta(3, 128), meta(3, 128), meta(3, 4, dt=F32), meta(3, dt=I32), meta(4, dt=F32)
    state, slots = meta(5, 4, 64, 32, dt=F32), meta(2, dt=I32)
    go = lambda **kw: wal.wal_delta(**dict(dict(desc=d, Q=q, K=q, V=v, A=g, B=g, starts=starts, out=v, state=state,  # noqa: E731
                                                slots=slots, decay=w, shift=w), **kw))
    for kw, err in ((dict(Q=meta(3, 120)), ValueError), (dict(K=meta(2, 128)), ValueError), (dict(V=meta(3, 128, dt=F32)), TypeError),
                    (dict(A=meta(3, 3, dt=F32)), ValueError), (dict(B=meta(3, 4)), TypeError), (dict(B=meta(2, 4, dt=F32)), ValueError),
                    (dict(state=None), ValueError), (dict(slots=None), ValueError), (dict(decay=None), ValueError),
                    (dict(shift=meta(3, dt=F32)), ValueError), (dict(state=meta(5, 4, 32, 64, dt=F32)), ValueError),
                    (dict(state=meta(5, 4, 64, 32)), TypeError), (dict(max_new=-1), ValueError), (dict(max_new=1 << 32), ValueError),
                    (dict(slots=meta(1, dt=I32)), ValueError), (dict(out=meta(2, 128)), ValueError),
                    (dict(Q=meta(3, 128, stride=((1 << 32) + 128, 1))), ValueError)):
        with pytest.raises(err):
            go(**kw)
    with pytest.raises(ValueError, match="GPU"):
        go()
    for bad in ((1 << 32, 1, 1), (1, -1, 1), (1, 1, 1 << 33)):
        with pytest.raises(ValueError, match="32 bits"):
            wal.wal_delta_workspace_size(d, *bad)
