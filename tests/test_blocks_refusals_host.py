"""More of what the calls of test_blocks_host.py refuse, without a GPU."""
import ctypes

import pytest
import torch

import ternary_hybrid_bit_amd as wal
from test_blocks_host import F32, I32, I64, meta

ARG, SHAPE, BUFFER, ALIGN = -1, -2, -5, -6


@pytest.mark.parametrize("rows", [0, 1, 3])
def test_rows_whose_elements_lie_apart(rows):
    """Refused however many rows there are."""
    far = meta(rows, 256, stride=(512, 2))
    near, w, pos, turns = meta(rows, 256), meta(64, dt=F32), meta(rows, dt=I32), meta(32, dt=I64)
    for call in (lambda: wal.wal_head_norm(far, near, w, 64), lambda: wal.wal_head_norm(near, far, w, 64),
                 lambda: wal.wal_rope(far, near, pos, turns, 64)):
        with pytest.raises(ValueError, match="unit stride"):
            call()
