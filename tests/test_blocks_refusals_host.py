"""More of what the binding and the library's calls of the blocks take and refuse, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import ternary_hybrid_bit_amd as wal
from test_blocks_host import F32, I32, I64, meta

ARG, SHAPE, BUFFER, ALIGN = -1, -2, -5, -6


def test_rows_whose_elements_lie_apart():
    """Refused where there are rows; tensors without any have the strides that their maker gave them (numpy: 0)."""
    assert torch.from_numpy(np.zeros((0, 256), np.float32)).stride() == (0, 0)
    w = meta(64, dt=F32)
    for rows, error in ((0, "GPU"), (1, "unit stride"), (3, "unit stride")):
        far, near = meta(rows, 256, stride=(512, 0)), meta(rows, 256)
        pos, turns = meta(rows, dt=I32), meta(32, dt=I64)
        for call in (lambda: wal.wal_head_norm(far, near, w, 64), lambda: wal.wal_head_norm(near, far, w, 64),
                     lambda: wal.wal_rope(far, near, pos, turns, 64)):
            with pytest.raises(ValueError, match=error):
                call()
