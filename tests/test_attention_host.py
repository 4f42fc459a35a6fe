"""Attention operators without a GPU: the host calls (wal_rope_freqs,
wal_kv_size, the workspace size), every check of arguments that comes before a
launch, the binding's own checks, and the float64 oracle on cases worked by
hand."""
import ctypes

import numpy as np
import pytest
import torch

import ternary_hybrid_bit_amd as wal
from oracle import attention as A

ARG, SHAPE, BUFFER, ALIGN = -1, -2, -5, -6


# ---- oracle ---------------------------------------------------------------

def test_oracle_rope_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    half, _ = A.rope(x, [1], [np.pi / 2, np.pi])
    np.testing.assert_allclose(half[0, 0], [-3, -2, 1, -4, 9], atol=1e-12)      # pairs (1,3) by 90, (2,4) by 180 degrees
    inter, _ = A.rope(x, [1], [np.pi / 2, np.pi], 2.0, interleaved=True)
    np.testing.assert_allclose(inter[0, 0], [-4, 2, -6, -8, 9], atol=1e-12)     # pairs (1,2), (3,4)


def test_oracle_rope_scores_depend_on_distance():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f, _ = A.rope_freqs(64, 10000.0)
    dot = [(A.rope(q, [p], f)[0] * A.rope(k, [p - 7], f)[0]).sum() for p in (7, 1000, 123456)]
    np.testing.assert_allclose(dot, dot[0], atol=1e-8)


def test_oracle_attend_by_hand():
    k = np.array([[[0.0]], [[0.0]], [[np.log(2.0)]]])
    v = np.array([[[1.0]], [[3.0]], [[8.0]]])
    out, size, _ = A.attend(np.ones((4, 1, 1)), k, v, [-1, 0, 1, 2], 1.0)
    np.testing.assert_allclose(out[:, 0, 0], [0, 1, 2, 5], atol=1e-12)          # weights 1/4, 1/4, 1/2 in the last
    out, _, _ = A.attend(np.ones((1, 1, 1)), k, v, [2], 1.0, present=[0, 0, 1])
    assert out[0, 0, 0] == 8.0


def test_oracle_int8_rows():
    c, s = A.int8_rows(np.array([[127.0, -63.5, 0.4, 0.0], [0, 0, 0, 0], [np.inf, 1, 2, 3], [np.nan, 1, 2, 3]]))
    assert c[0].tolist() == [127, -64, 0, 0] and s[0] == np.float32(127) * np.float32(1 / 127)
    assert s[1] == 0 and not c[1].any() and np.isnan(s[2]) and np.isnan(s[3])


# ---- host calls -----------------------------------------------------------

@pytest.mark.parametrize("rot", [16, 64, 96, 256])
@pytest.mark.parametrize("scaling", ["plain", "linear", "ntk", "parts"])
def test_rope_freqs(rot, scaling):
    factor = 1.0 if scaling == "plain" else 8.0
    code = {"plain": 0, "linear": 1, "ntk": 2, "parts": 3}[scaling]
    turns, m = wal.wal_rope_freqs(wal.make_rope_desc(rot, 1e6, code, factor, 4096.0, 1.0, 32.0))
    f, magnitude = A.rope_freqs(rot, 1e6, scaling, factor, 4096.0, 1.0, 32.0)
    assert turns.shape == (rot // 2,) and m == np.float32(magnitude)
    # the table holds the nearest whole number of units of 2^-64 turns: half a unit, and float64's pow and
    # products, a few 2^-52 of the value on either side
    units = 2.0 ** 64 * f / (2 * np.pi)
    assert (np.abs(turns.astype(np.float64) - units) <= 0.5 + 2.0 ** -48 * units).all()


def test_rope_freqs_rejects():
    lib, t = wal._lib, np.zeros(256, np.int64)
    ok = dict(rot_dim=64, base=1e4, scaling=0, factor=1.0)
    call = lambda turns=t.ctypes.data, **kw: lib.wal_rope_freqs(  # noqa: E731
        ctypes.byref(wal.make_rope_desc(**{**ok, **kw})), turns, None)
    assert call() == 0
    assert call(turns=None) == ARG and lib.wal_rope_freqs(None, t.ctypes.data, None) == ARG
    assert [call(rot_dim=r) for r in (0, 8, 24, 528)] == [SHAPE] * 4
    assert [call(base=b) for b in (1.0, 0.0, -2.0, float("nan"), float("inf"))] == [ARG] * 5
    assert call(scaling=4) == ARG
    assert [call(scaling=1, factor=f) for f in (0.5, float("nan"), float("inf"))] == [ARG] * 3
    parts = dict(scaling=3, factor=2.0, trained_len=4096.0)
    assert call(**parts) == 0 and call(**{**parts, "trained_len": 0.0}) == ARG
    assert call(**parts, turns_low=32.0, turns_high=32.0) == ARG and call(**parts, turns_low=-1.0) == ARG


def test_kv_size():
    f = wal.wal_kv_size(wal.make_kv_desc(3, 16, 5, 64, wal.WAL_KV_BF16))
    plane = 3 * 16 * 5 * 64 * 2
    assert plane % 256 == 0 and (f.off_k, f.off_v, f.total_bytes) == (0, plane, 2 * plane)
    f = wal.wal_kv_size(wal.make_kv_desc(1, 16, 1, 64, wal.WAL_KV_INT8))
    assert (f.off_k, f.off_v, f.off_ks, f.off_vs, f.total_bytes) == (0, 1024, 2048, 2304, 2560)   # 64-byte scale planes
    big = wal.wal_kv_size(wal.make_kv_desc(1 << 23, 256, 8, 128, wal.WAL_KV_BF16))
    assert big.off_v == (1 << 31) * 8 * 128 * 2
    for bad in [(0, 16, 1, 64, 0), (1, 24, 1, 64, 0), (1, 8, 1, 64, 0), (1, 512, 1, 64, 0), (1, 16, 0, 64, 0),
                (1, 16, 257, 64, 0), (1, 16, 1, 96, 0), (1 << 24, 256, 1, 64, 0)]:
        with pytest.raises(wal.WalError) as e:
            wal.wal_kv_size(wal.make_kv_desc(*bad))
        assert e.value.status == SHAPE, bad
    with pytest.raises(wal.WalError) as e:
        wal.wal_kv_size(wal.make_kv_desc(1, 16, 1, 64, 2))
    assert e.value.status == ARG
    assert wal._lib.wal_kv_size(None, ctypes.byref(f)) == ARG
    assert wal._lib.wal_kv_size(ctypes.byref(wal.make_kv_desc(1, 16, 1, 64)), None) == ARG


# ---- checks before any launch (the pointers are never read) ----------------

X, Y, T, P, C, S, K, V, Q, O, W = (0x10000000 * i for i in range(1, 12))


def rot(turns=T, pos=P, dim=64, layout=0):
    return ctypes.byref(wal.wal_rotary(turns, pos, dim, layout, 1.0))


def test_rope_checks():
    f = wal._lib.wal_rope
    assert f(X, 1, 0, 4, 64, 256, rot(), Y, 1, 256, None) == 0                      # no token: nothing to do
    assert f(None, 1, 2, 4, 64, 256, rot(), Y, 1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 256, None, Y, 1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 256, rot(), None, 1, 256, None) == ARG
    assert f(X, 2, 2, 4, 64, 256, rot(), Y, 1, 256, None) == ARG                    # dtypes
    assert f(X, 1, 2, 4, 64, 256, rot(), Y, -1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 255, rot(), Y, 1, 256, None) == ARG                    # pitch below the width
    assert f(X, 1, 2, 4, 64, 260, rot(), Y, 1, 256, None) == ALIGN                  # rows not 16-byte aligned
    assert f(X + 8, 1, 2, 4, 64, 256, rot(), Y, 1, 256, None) == ALIGN
    assert f(X, 1, 2, 0, 64, 256, rot(), Y, 1, 256, None) == SHAPE
    assert [f(X, 1, 2, 4, d, 4096, rot(), Y, 1, 4096, None) for d in (0, 72, 528)] == [SHAPE] * 3
    assert [f(X, 1, 2, 4, 64, 256, rot(dim=d), Y, 1, 256, None) for d in (0, 8, 40, 80)] == [SHAPE] * 4
    assert f(X, 1, 2, 4, 64, 256, rot(layout=2), Y, 1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 256, rot(turns=None), Y, 1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 256, rot(pos=None), Y, 1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 256, rot(turns=T + 4), Y, 1, 256, None) == ALIGN
    assert f(X, 1, 2, 4, 64, 256, rot(pos=P + 2), Y, 1, 256, None) == ALIGN
    assert f(X, 1, 2, 4, 64, 256, rot(), X + 512, 1, 256, None) == ARG              # overlaps x
    assert f(X, 1, 2, 4, 64, 256, rot(), X, 0, 256, None) == ARG                    # in place with another type
    assert f(X, 1, 2, 4, 64, 256, rot(pos=Y), Y, 1, 256, None) == ARG
    assert f(X, 1, 2, 4, 64, 256, rot(turns=Y + 256), Y, 1, 256, None) == ARG


def test_kv_write_checks():
    d = wal.make_kv_desc(4, 16, 2, 64, 1)

    def f(desc=ctypes.byref(d), c=C, s=S, n=3, k=K, ldk=128, v=V, ldv=128, t=1, r=rot(), q=Q, h=4, ldq=256, o=O,
          ldo=256):
        return wal._lib.wal_kv_write(desc, c, s, n, k, ldk, v, ldv, t, r, q, h, ldq, o, ldo, None)
    assert f(n=0) == 0
    assert [f(desc=None), f(c=None), f(s=None), f(k=None), f(v=None), f(t=2), f(o=None), f(q=None)] == [ARG] * 8
    assert f(r=None) == ARG                                  # q without a rotation
    assert f(ldk=120) == ARG and f(ldq=248) == ARG and f(ldo=248) == ARG
    assert f(ldk=132) == ALIGN and f(c=C + 128) == ALIGN and f(s=S + 2) == ALIGN and f(q=Q + 4) == ALIGN
    assert f(h=0) == SHAPE and f(r=rot(dim=128)) == SHAPE
    assert f(k=C + 1024) == ARG and f(o=C) == ARG and f(o=K) == ARG and f(s=C) == ARG and f(q=C) == ARG
    assert f(o=Q + 16) == ARG                                # q_out overlaps q
    bad = wal.make_kv_desc(4, 20, 2, 64, 1)
    assert f(desc=ctypes.byref(bad)) == SHAPE


def test_kv_read_checks():
    d = wal.make_kv_desc(4, 16, 2, 64, 0)

    def f(desc=ctypes.byref(d), c=C, s=S, n=3, k=K, ldk=128, v=V, ldv=128, t=1):
        return wal._lib.wal_kv_read(desc, c, s, n, k, ldk, v, ldv, t, None)
    assert f(n=0) == 0
    assert [f(desc=None), f(c=None), f(s=None), f(k=None, v=None), f(t=3), f(ldk=127), f(v=K + 16)] == [ARG] * 7
    assert f(k=C + 256) == ARG and f(v=S) == ARG
    assert f(ldv=129) == ALIGN and f(k=K + 2) == ALIGN and f(c=C + 16) == ALIGN


def test_attn_paged_checks():
    d = wal.make_kv_desc(8, 16, 2, 64, 0)
    lib = wal._lib

    def size(desc=d, h=4, seqs=2, n=3, new=2, most=64):
        b = ctypes.c_size_t()
        st = lib.wal_attn_paged_workspace_size(ctypes.byref(desc), h, seqs, n, new, most, ctypes.byref(b))
        return st or b.value
    need = size()

    def f(desc=ctypes.byref(d), c=C, t=T, ldt=4, l=P, s=S, seqs=2, n=3, new=2, most=64, q=Q, h=4, ldq=256, scale=0.1,
          o=O, ldo=256, w=W, wb=1 << 24):
        return lib.wal_attn_paged(desc, c, t, ldt, l, s, seqs, n, new, most, q, h, ldq, scale, o, ldo, w, wb, None)
    assert f(n=0) == 0 and f(seqs=0) == 0 and f(new=0) == 0
    assert [f(desc=None), f(c=None), f(t=None), f(l=None), f(s=None), f(q=None), f(o=None)] == [ARG] * 7
    assert f(scale=float("nan")) == ARG and f(scale=float("inf")) == ARG
    assert f(scale=3e38) == ARG                              # infinite times log2(e)
    assert f(ldt=3) == ARG                                   # the tables do not hold max_len tokens
    assert f(h=3) == SHAPE and f(h=0) == SHAPE and f(h=2 * 65, ldq=8320, ldo=8320) == SHAPE
    assert f(ldq=248) == ARG and f(ldq=260) == ALIGN and f(q=Q + 8) == ALIGN and f(c=C + 16) == ALIGN
    assert f(l=P + 1) == ALIGN and f(s=S + 2) == ALIGN and f(t=T + 2) == ALIGN
    assert f(o=Q) == ARG and f(o=C) == ARG and f(o=T) == ARG and f(o=P) == ARG and f(o=S) == ARG
    assert size(h=3) == SHAPE and size(n=(1 << 24) + 1) == SHAPE and size(most=(1 << 30) + 1) == SHAPE
    assert size(h=128, n=1 << 24) == SHAPE                   # n * q_heads
    many = size(seqs=1, n=1, new=1, most=128)
    assert many >= 0 and need >= 0
    split = wal.wal_attn_paged_workspace_size(wal.make_kv_desc(8192, 16, 2, 64, 0), 4, 1, 1, 1, 131072)
    if split:                                                # a long context is split: the workspace is needed
        big = wal.make_kv_desc(8192, 16, 2, 64, 0)
        long = dict(desc=ctypes.byref(big), ldt=8192, seqs=1, n=1, new=1, most=131072)
        assert f(**long, wb=split - 1) == BUFFER and f(**long, w=None) == ARG and f(**long, w=W + 128) == ALIGN
        assert f(**long, w=O) == ARG and f(**long, w=C) == ARG


def test_attn_prompt_checks():
    def f(q=Q, ldq=256, k=K, ldk=128, v=V, ldv=128, s=S, seqs=2, n=3, most=2, h=4, kvh=2, d=64, scale=0.1, o=O,
          ldo=256):
        return wal._lib.wal_attn_prompt(q, ldq, k, ldk, v, ldv, s, seqs, n, most, h, kvh, d, scale, 1, o, ldo, None)
    assert f(n=0) == 0 and f(seqs=0) == 0 and f(most=0) == 0
    assert [f(q=None), f(k=None), f(v=None), f(s=None), f(o=None), f(scale=float("nan"))] == [ARG] * 6
    assert f(h=3) == SHAPE and f(kvh=0) == SHAPE and f(d=96) == SHAPE and f(h=0) == SHAPE
    assert f(ldq=255) == ARG and f(ldk=124) == ARG and f(ldv=132) == ALIGN and f(k=K + 8) == ALIGN
    assert f(s=S + 2) == ALIGN
    assert f(o=Q) == ARG and f(o=K) == ARG and f(o=V) == ARG and f(o=S) == ARG


def test_columns_of_one_buffer_do_not_overlap():
    """q, k, v and the output side by side in rows of one buffer are accepted (n = 0 launches nothing; the
    overlap check runs before), rows that share a column are not."""
    f = wal._lib.wal_kv_write
    d = wal.make_kv_desc(4, 16, 2, 64, 0)
    assert f(ctypes.byref(d), C, S, 0, X + 512, 512, X + 768, 512, 1, rot(), X, 4, 512, X, 512, None) == 0
    bad = (ctypes.byref(d), C, S, 3, X + 256, 512, X + 768, 512, 1, rot(), X, 4, 512, X, 512, None)
    assert f(*bad) == ARG                                    # k's columns lie in q's, which is rotated in place


# ---- the binding's own checks ----------------------------------------------

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def z(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


def test_binding_rope():
    pos, turns = z(3, dt=I32), z(32, dt=torch.int64)
    with pytest.raises(ValueError):
        wal.wal_rope(z(3, 200), z(3, 200), pos, turns, 64)              # not whole heads
    with pytest.raises(ValueError):
        wal.wal_rope(z(3, 256), z(2, 256), pos, turns, 64)              # short output
    with pytest.raises(TypeError):
        wal.wal_rope(z(3, 256), z(3, 256), pos.long(), turns, 64)
    with pytest.raises(TypeError):
        wal.wal_rope(z(3, 256), z(3, 256), pos, turns.double(), 64)
    with pytest.raises(ValueError):
        wal.wal_rope(z(3, 256), z(3, 256), pos[:2], turns, 64)
    with pytest.raises(TypeError):
        wal.wal_rope(z(3, 256, dt=torch.float16), z(3, 256), pos, turns, 64)
    with pytest.raises(ValueError, match="GPU"):
        wal.wal_rope(z(3, 256), z(3, 256), pos, turns, 64)


def test_binding_cache():
    d = wal.make_kv_desc(2, 16, 2, 64)
    n = wal.wal_kv_size(d).total_bytes
    cache, slots, k = z(n, dt=torch.uint8), z(3, dt=I32), z(3, 128)
    pos, turns = z(3, dt=I32), z(32, dt=torch.int64)
    with pytest.raises(ValueError):
        wal.wal_kv_write(d, cache[:-1], slots, k, k)
    with pytest.raises(ValueError):
        wal.wal_kv_write(d, cache, slots[:2], k, k)
    with pytest.raises(TypeError):
        wal.wal_kv_write(d, cache, slots, k, k.float())                 # k and v of one type
    with pytest.raises(ValueError):
        wal.wal_kv_write(d, cache, slots, z(3, 64), k)
    with pytest.raises(ValueError):
        wal.wal_kv_write(d, cache, slots, k, k, pos=pos)
    with pytest.raises(ValueError):
        wal.wal_kv_write(d, cache, slots, k, k, pos=pos, turns=turns, Q=z(3, 256))
    with pytest.raises(TypeError):
        wal.wal_kv_write(d, cache, slots, k, k, pos=pos, turns=turns, Q=z(3, 256), Q_out=z(3, 256, dt=F32))
    with pytest.raises(ValueError, match="GPU"):
        wal.wal_kv_write(d, cache, slots, k, k, pos=pos, turns=turns, Q=z(3, 256), Q_out=z(3, 256))
    with pytest.raises(ValueError):
        wal.wal_kv_read(d, cache, slots)
    with pytest.raises(ValueError):
        wal.wal_kv_read(d, cache, slots, K=z(2, 128))
    with pytest.raises(TypeError):
        wal.wal_kv_read(d, cache, slots, K=z(3, 128), V=z(3, 128, dt=F32))
    with pytest.raises(ValueError, match="GPU"):
        wal.wal_kv_read(d, cache, slots, V=z(3, 128))


def test_binding_attention():
    d = wal.make_kv_desc(2, 16, 2, 64)
    cache = z(wal.wal_kv_size(d).total_bytes, dt=torch.uint8)
    tables, lens, starts = z(2, 1, dt=I32), z(2, dt=I32), z(3, dt=I32)
    q = z(4, 256)
    ok = dict(desc=d, cache=cache, tables=tables, lens=lens, starts=starts, Q=q, out=z(4, 256))
    for kw, err in [(dict(tables=tables.long()), TypeError), (dict(lens=lens[:1]), ValueError),
                    (dict(starts=starts[:2]), ValueError), (dict(Q=q.float()), TypeError),
                    (dict(out=z(3, 256)), ValueError), (dict(Q=z(4, 200)), ValueError), (dict(max_len=17), ValueError),
                    (dict(max_new=-1), ValueError), (dict(cache=cache[1:]), ValueError)]:
        with pytest.raises(err):
            wal.wal_attn_paged(**{**ok, **kw})
    with pytest.raises(ValueError, match="GPU"):
        wal.wal_attn_paged(**ok)
    k = z(4, 128)
    for a, err in [((q, k, k[:3], starts, z(4, 256)), ValueError), ((q, k, z(4, 64), starts, z(4, 256)), ValueError),
                   ((q, k, k, starts.long(), z(4, 256)), TypeError), ((q, k, k, starts, z(4, 128)), ValueError)]:
        with pytest.raises(err):
            wal.wal_attn_prompt(*a, 64, 4)
    with pytest.raises(ValueError, match="GPU"):
        wal.wal_attn_prompt(q, k, k, starts, z(4, 256), 64, 4)
