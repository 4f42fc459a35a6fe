"""GPU tests of the attention operators where arguments or contents are out of the ordinary; the helpers and
tolerances are those of test_gpu_attention.py."""
import numpy as np
import pytest

from test_gpu_attention import BF16, INT8, Paged, dev, host, i32, table, wal  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LO, HI = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("starts", [(5, LO, 8), (HI, LO, 8), (HI, -2, HI), (5, LO + 7, LO), (0, HI, LO), (LO, LO, LO),
                                    (8, HI, HI), (3, -1, 6)])
@pytest.mark.parametrize("max_new", [1, 4])
def test_extreme_starts_stay_inside(wal, starts, max_new):  # noqa: F811
    """starts at the ends of int32: rows around the output keep what they hold (the host test of the same cutting goes
    over many more values)."""
    print(f"starts {starts} max_new {max_new}", flush=True)
    p = Paged(wal, [(100, 4), (60, 4)], 4, 2, 128, 16, BF16, seed=17)
    wide = torch.full((24, 1024), 77.0, dtype=torch.bfloat16, device=dev())
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev())
    for lens in ([100, 60], [HI, LO], [LO, HI]):
        wal.wal_attn_paged(p.d, p.cache, i32(p.tables), i32(lens), i32(starts), p.Q, wide[8:16], ws, max_new=max_new,
                           max_len=100)
        wal.wal_attn_prompt(p.Q, p.Q[:, :256], p.Q[:, 256:512], i32(starts), wide[8:16], 128, 4)
    torch.cuda.synchronize()
    assert (wide[:8] == 77.0).all() and (wide[16:] == 77.0).all()
    assert not ws[:wal.WAL_ATTN_WS_ZERO_BYTES].any()


@pytest.mark.parametrize("fmt", [BF16, INT8])
@pytest.mark.parametrize("n,new,dim", [(200, 1, 128), (200, 1, 64), (200, 4, 256), (200, 7, 128), (200, 50, 128),
                                       (2900, 1, 128), (2900, 30, 64)])
@pytest.mark.parametrize("where", ["seen by all", "seen by some"])
def test_nan_of_a_weight_that_underflows(wal, fmt, n, new, dim, where):  # noqa: F811
    """One key takes all the weight: a seen value row that is NaN makes its rows NaN though its weight is 0 in fp32, in
    every kernel; rows that do not see it stay numbers."""
    print(f"n={n} new={new} dim={dim} fmt={fmt} {where}", flush=True)
    p = Paged(wal, [(n, new), (80, 1)], 4, 1, dim, 16, fmt, seed=31)
    p.Q[:] = p.Q[:1, :dim].repeat(p.Q.shape[0], 4)                 # every row and head asks the same
    # in one tile of the kernels for few rows, so that the same wavefront holds the maximum
    bad = 20 if where == "seen by all" else n - new // 2 - 1
    hot = min(bad - 2, n - new)
    K = torch.cat([p.Q[:1, :dim].float() * 40, torch.zeros((1, dim), device=dev())])   # a score of 40 sqrt(dim): > 300
    V = torch.ones((2, dim), device=dev())
    V[1, 5] = float("nan")
    wal.wal_kv_write(p.d, p.cache, p.slots[[hot, bad]].contiguous(), K, V)
    got = host(p.call()).reshape(-1, 4, dim)
    sees = np.append(n - new + np.arange(new) >= bad, False)
    assert sees.any()
    nan = np.isnan(got[sees]) if fmt == INT8 else np.isnan(got[sees][..., 5:6])   # int8: the whole row's scale
    assert nan.all() and np.isfinite(got[~sees]).all()
    assert (got[:new][~sees[:new]] == 1.0).all()                   # the hot key's value


@pytest.mark.parametrize("seqs", [[(300, 40)], [(90, 5), (40, 1)], [(64, 64), (0, 0), (7, 7)], [(200, 1), (33, 1)]])
def test_max_new_left_out(wal, seqs):  # noqa: F811
    """Every row is computed when the call is not told how many new tokens the sequences have."""
    p = Paged(wal, seqs, 4, 2, 128, 16, BF16, seed=41)
    p.call()                                   # (makes the arguments)
    n = p.Q.shape[0]
    ws = torch.zeros(max(wal.WAL_ATTN_WS_ZERO_BYTES, wal.wal_attn_paged_workspace_size(
        p.d, 8, len(seqs), n, n, p.tables.shape[1] * 16)), dtype=torch.uint8, device=dev())
    out = torch.full((n, p.Q.shape[1]), 77.0, dtype=torch.bfloat16, device=dev())
    wal.wal_attn_paged(p.d, p.cache, *p.args, p.Q, out, ws)
    p.check(out)


def test_the_pitch_of_an_only_row_means_nothing(wal):  # noqa: F811
    """One token in buffers whose rows are not 16 bytes apart: there is no second row."""
    heads, dim, n = 2, 64, 1

    def row(cols, dtype=torch.bfloat16):
        t = torch.randn((3, cols + 3), device=dev()).to(dtype)[:1, :cols]
        assert t.stride(0) == cols + 3 and t.data_ptr() % 16 == 0
        return t
    turns, _, m = table(wal, dim, "plain", 1.0)
    pos, slots = i32([7]), i32([5])
    d = wal.make_kv_desc(2, 16, heads, dim, BF16)
    for dtype in (torch.bfloat16, torch.float32):
        q, k, v = row(4 * dim, dtype), row(2 * dim, dtype), row(2 * dim, dtype)
        results = []
        for wrap in (lambda t: t, lambda t: t.contiguous()):
            a, b, c = wrap(q), wrap(k), wrap(v)
            turned, q_out, k2, v2, out, whole = (wrap(row(w, t)) for w, t in (
                (4 * dim, dtype), (4 * dim, torch.bfloat16), (2 * dim, dtype), (2 * dim, dtype), (4 * dim, torch.bfloat16),
                (4 * dim, torch.bfloat16)))
            cache = torch.zeros(wal.wal_kv_size(d).total_bytes, dtype=torch.uint8, device=dev())
            wal.wal_rope(a, turned, pos, turns, dim)
            wal.wal_kv_write(d, cache, slots, b, c, pos=pos, turns=turns, Q=a, Q_out=q_out)
            wal.wal_kv_read(d, cache, slots, k2, v2)
            wal.wal_attn_paged(d, cache, torch.zeros((3, 5), dtype=torch.int32, device=dev())[:1, :2], i32([6]), i32([0, n]),
                               q_out, out, max_len=32)
            wal.wal_attn_prompt(q_out, k2.to(torch.bfloat16), v2.to(torch.bfloat16), i32([0, n]), whole, dim, 1)
            results.append([turned, q_out, k2, v2, out, whole])
            assert all(torch.isfinite(t).all() for t in results[-1])
        assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("n,new,dim", [(120, 1, 128), (120, 7, 128), (120, 60, 64), (5000, 1, 64), (5000, 40, 128)])
def test_rows_whose_scores_are_all_minus_infinity(wal, n, new, dim):  # noqa: F811
    p = Paged(wal, [(n, new), (40, 1)], 4, 2, dim, 16, BF16, seed=51)
    p.Q[:, 5::dim] = 1.0
    K, V = (torch.from_numpy(x[:n].reshape(n, -1).astype(np.float32)).to(dev()) for x in (p.k, p.v))
    K[:, 5] = float("-inf")                    # the first key/value head of the first sequence
    wal.wal_kv_write(p.d, p.cache, p.slots[:n].contiguous(), K, V)
    got = host(p.call()).reshape(-1, 2, 4, dim)
    assert (got[:new, 0] == 0).all() and np.isfinite(got).all() and (got[new:] != 0).any() and (got[:new, 1] != 0).any()
