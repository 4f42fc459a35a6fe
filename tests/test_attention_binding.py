"""Sizes that the library's 32-bit arguments cannot hold are refused by the binding, not cut to their low
bits; tensors on torch's meta device stand for those that no machine here holds."""
import pytest
import torch

import ternary_hybrid_bit_amd as wal

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


def meta(*shape, dt=BF, stride=None):
    stride = stride or tuple(int(torch.tensor(shape[i + 1:]).prod()) for i in range(len(shape)))
    return torch.empty_strided(shape, stride, dtype=dt, device="meta")


def test_pitches_past_32_bits():
    far = meta(2, 256, stride=((1 << 32) + 256, 1))
    near = meta(2, 256)
    pos, turns, slots, starts = meta(2, dt=I32), meta(32, dt=I64), meta(2, dt=I32), meta(2, dt=I32)
    d = wal.make_kv_desc(1, 16, 4, 64)
    cache = meta(wal.wal_kv_size(d).total_bytes, dt=torch.uint8)
    tables, lens = meta(2, 1, dt=I32), meta(2, dt=I32)
    for call in (lambda x, y: wal.wal_rope(x, y, pos, turns, 64),
                 lambda x, y: wal.wal_kv_write(d, cache, slots, x, y),
                 lambda x, y: wal.wal_kv_write(d, cache, slots, y, near, pos=pos, turns=turns, Q=x, Q_out=near),
                 lambda x, y: wal.wal_kv_read(d, cache, slots, x, y),
                 lambda x, y: wal.wal_attn_paged(d, cache, tables, lens, meta(3, dt=I32), x, y),
                 lambda x, y: wal.wal_attn_prompt(x, y, near, starts, near, 64, 2),
                 lambda x, y: wal.wal_attn_prompt(near, near, x, starts, y, 64, 2)):
        for x, y in ((far, near), (near, far)):
            with pytest.raises(ValueError, match="32 bits"):
                call(x, y)
        with pytest.raises(ValueError, match="GPU"):
            call(near, near)
    with pytest.raises(ValueError, match="32 bits"):
        wal.wal_attn_paged(d, cache, meta(2, 1, dt=I32, stride=(1 << 32, 1)), lens, meta(3, dt=I32), near, near)


def test_rows_past_32_bits():
    n = (1 << 32) + 2
    x = meta(n, 256)
    with pytest.raises(ValueError, match="32 bits"):
        wal.wal_rope(x, x, meta(n, dt=I32), meta(32, dt=I64), 64)
    d = wal.make_kv_desc(1, 16, 4, 64)
    cache = meta(wal.wal_kv_size(d).total_bytes, dt=torch.uint8)
    with pytest.raises(ValueError, match="32 bits"):
        wal.wal_kv_read(d, cache, meta(n, dt=I32), x)
    with pytest.raises(ValueError, match="32 bits"):
        wal.wal_attn_prompt(meta(2, 256), meta(2, 256), meta(2, 256), meta(n, dt=I32), meta(2, 256), 64, 2)


@pytest.mark.parametrize("bound", [1 << 32, (1 << 32) + 1, -1])
def test_bounds_past_32_bits(bound):
    d = wal.make_kv_desc(1, 16, 4, 64)
    cache = meta(wal.wal_kv_size(d).total_bytes, dt=torch.uint8)
    q = meta(2, 256)
    with pytest.raises(ValueError, match="max_new"):
        wal.wal_attn_paged(d, cache, meta(2, 1, dt=I32), meta(2, dt=I32), meta(3, dt=I32), q, q, max_new=bound)
    with pytest.raises(ValueError, match="max_len"):
        wal.wal_attn_prompt(q, q, q, meta(2, dt=I32), q, 64, bound)
    for args in () if bound < 0 else ((4, 1, 2, 1, bound), (4, 1, 2, bound, 16), (4, 1, bound, 1, 16), (4, bound, 2, 1, 16), (bound, 1, 2, 1, 16)):
        with pytest.raises(ValueError, match="32 bits"):
            wal.wal_attn_paged_workspace_size(d, *args)
