"""GPU tests of calls that need more workgroups than a launch can have (2^24 of 256 threads): rows at both ends of a call
are done, bit for bit as in a short one."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wal():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import ternary_hybrid_bit_amd as w
    return w


def test_cache_write_of_more_rows_than_a_launch_takes(wal):
    """One token a workgroup (136 units of it), 2^24 + 5 tokens, all but a few outside the cache; 36 GB, not initialised."""
    n, heads, dim = (1 << 24) + 5, 17, 64
    desc = wal.make_kv_desc(2, 16, heads, dim)
    rows = torch.tensor([0, 1, (1 << 23) + 1, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, n - 1], device="cuda")
    few = torch.randn((len(rows), heads * dim), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    cache, want = (torch.zeros(wal.wal_kv_size(desc).total_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    place = torch.arange(len(rows), dtype=torch.int32, device="cuda") * 4
    wal.wal_kv_write(desc, want, place, few, few)
    x = torch.empty((n, heads * dim), dtype=torch.bfloat16, device="cuda")
    x[rows] = few
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[rows] = place
    wal.wal_kv_write(desc, cache, slots, x, x)
    torch.cuda.synchronize()
    assert want.any() and torch.equal(cache, want)
    del x
    torch.cuda.empty_cache()


def test_rotation_of_more_rows_than_a_launch_takes(wal):
    """2^24 + 3 rows of one group (4.3 GB, in place)."""
    n = (1 << 24) + 3
    rows = torch.tensor([0, 5, 1 << 23, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, n - 1], device="cuda")
    few = torch.randn((len(rows), 128), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    want = torch.empty_like(few)
    wal.wal_rotate_h128(few, want)
    x = torch.empty((n, 128), dtype=torch.bfloat16, device="cuda")
    x[rows] = few
    wal.wal_rotate_h128(x, x)
    torch.cuda.synchronize()
    assert torch.equal(x[rows], want) and not torch.equal(few, want)


@pytest.mark.parametrize("mixed", [False, True])
def test_embedding_of_more_tokens_than_a_launch_takes(wal, mixed):
    """2^25 + 3 tokens of 128 columns (8.6 GB)."""
    import numpy as np
    rng, V = np.random.default_rng(4), 16
    pack = lambda bits: torch.from_numpy((wal.wal_int3_pack if bits == 3 else wal.wal_int4_pack)(  # noqa: E731
        rng.integers(-4, 4, (V, 128)).astype(np.int8), rng.uniform(0.1, 1, (V, 1)).astype(np.float16).astype(np.float32))).cuda()
    W3, W4 = pack(3), pack(4)
    n = (1 << 25) + 3
    ids = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    row_map = torch.tensor([v if v % 2 else -1 - v for v in range(V)], dtype=torch.int32, device="cuda")
    embed = (lambda i, o: wal.wal_embed_rows_mixed(W3, V, W4, V, 128, row_map, i, o)) if mixed else (  # noqa: E731
        lambda i, o: wal.wal_embed_rows(W3, 3, V, 128, i, o))
    out = torch.full((n, 128), -9.0, dtype=torch.bfloat16, device="cuda")
    embed(ids, out)
    for part in (slice(0, 4), slice((1 << 25) - 4, n), slice(1 << 24, (1 << 24) + 4)):
        want = torch.empty((ids[part].numel(), 128), dtype=torch.bfloat16, device="cuda")
        embed(ids[part].clone(), want)
        assert torch.equal(out[part], want) and (want != -9).any()


def test_delta_rule_of_more_sequences_than_a_launch_takes(wal):
    """1024 heads of 256 columns, 2^13 sequences of which three bring a token: 2^25 workgroups."""
    seqs, n, h, dk, dv = 1 << 13, 3, 1024, 64, 256
    desc = wal.make_delta_desc(h, h, dk, dv)
    g = torch.Generator("cuda").manual_seed(2)
    q, k = (torch.randn((n, h * dk), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    v = torch.randn((n, h * dv), device="cuda", generator=g).to(torch.bfloat16)
    a, b = -torch.rand((n, h), device="cuda", generator=g), torch.rand((n, h), device="cuda", generator=g)
    starts = torch.zeros(seqs + 1, dtype=torch.int32)
    starts[1:] += 1
    starts[seqs // 2:] += 1
    starts[seqs:] += 1
    few = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    want, out = (torch.full((n, h * dv), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wal.wal_delta(desc, q, k, v, a, b, few.cuda(), want, max_new=1)
    wal.wal_delta(desc, q, k, v, a, b, starts.cuda(), out, max_new=1)
    torch.cuda.synchronize()
    assert (want != -7).all() and torch.equal(out, want)


def test_delta_rule_of_rows_far_apart(wal):
    """The largest pitch, 2^24 elements, on chunks (2.3 GB each for v and the outputs)."""
    n, h, dk, dv, far = 70, 2, 64, 64, 1 << 24
    desc = wal.make_delta_desc(h, h, dk, dv)
    g = torch.Generator("cuda").manual_seed(6)
    q, k, v = (torch.randn((n, h * d), device="cuda", generator=g).to(torch.bfloat16) for d in (dk, dk, dv))
    a, b = -torch.rand((n, h), device="cuda", generator=g), torch.rand((n, h), device="cuda", generator=g)
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ws = torch.empty(wal.wal_delta_workspace_size(desc, 1, n, n), dtype=torch.uint8, device="cuda")
    want = torch.empty((n, h * dv), dtype=torch.bfloat16, device="cuda")
    wal.wal_delta(desc, q, k, v, a, b, starts, want, ws=ws)
    wide, out = (torch.empty((n, far), dtype=torch.bfloat16, device="cuda")[:, 8:8 + h * dv] for _ in range(2))
    wide.copy_(v)
    wal.wal_delta(desc, q, k, wide, a, b, starts, out, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.isfinite(want).all()
