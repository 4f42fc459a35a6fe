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
