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
