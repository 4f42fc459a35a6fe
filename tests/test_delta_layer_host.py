"""What DeltaLayer refuses before it is built, without a GPU: a tensor or number that one of its calls would refuse later,
between the launches that change its states."""
import types

import pytest
import torch

from ternary_hybrid_bit_amd.delta import DeltaLayer

KH, VH, DK, DV = 2, 4, 64, 32
CHANNELS = 2 * KH * DK + VH * DV
BF = torch.bfloat16


def matrix(rows, cols=512):
    return types.SimpleNamespace(d=types.SimpleNamespace(out=rows, in_=cols)), torch.zeros(1, dtype=torch.uint8)


def layer(**kw):
    small = dict(conv=torch.zeros((CHANNELS, 4)), decay=torch.ones(VH), shift=torch.zeros(VH), norm=torch.ones(DV))
    sizes = dict(key_heads=KH, value_heads=VH, key_dim=DK, value_dim=DV, max_seqs=2)
    return DeltaLayer(matrix(CHANNELS), matrix(VH * DV), matrix(2 * VH), matrix(512, VH * DV), **dict(small, **sizes, **kw))


def test_what_it_takes():
    assert layer().rows.shape == (2, 3, CHANNELS) and layer().state.shape == (2, VH, DK, DV)
    assert layer(conv=torch.zeros((CHANNELS, 2), dtype=BF), conv_bias=torch.zeros(CHANNELS, dtype=BF),
                 norm=torch.ones(DV, dtype=BF)).rows.shape[1] == 1


@pytest.mark.parametrize("kw,err", [
    (dict(decay=torch.ones(VH, dtype=BF)), TypeError), (dict(decay=torch.ones(VH - 1)), ValueError), (dict(decay=None), TypeError),
    (dict(decay=torch.ones(2 * VH)[::2]), ValueError), (dict(shift=torch.zeros(VH, dtype=torch.float64)), TypeError),
    (dict(shift=torch.zeros((VH, 1))), ValueError), (dict(norm=torch.ones(DV + 1)), ValueError), (dict(norm=[1.0] * DV), TypeError),
    (dict(norm=torch.ones(DV, dtype=torch.float16)), TypeError), (dict(norm=torch.ones(2 * DV)[::2]), ValueError),
    (dict(conv=torch.zeros((CHANNELS - 8, 4))), ValueError), (dict(conv=torch.zeros((CHANNELS, 5))), ValueError),
    (dict(conv=torch.zeros((CHANNELS, 1))), ValueError), (dict(conv=torch.zeros((4, CHANNELS)).t()), ValueError),
    (dict(conv=torch.zeros((CHANNELS, 4), dtype=torch.float16)), TypeError), (dict(conv=torch.zeros(CHANNELS * 4)), ValueError),
    (dict(conv=torch.zeros(CHANNELS * 4 + 1)[1:].view(CHANNELS, 4)), ValueError),
    (dict(conv_bias=torch.zeros(CHANNELS, dtype=BF)), TypeError), (dict(conv_bias=torch.zeros(CHANNELS - 1)), ValueError),
    (dict(norm=torch.ones(DV, device="meta")), ValueError), (dict(eps=0.0), ValueError), (dict(eps=float("nan")), ValueError),
    (dict(eps=float("inf")), ValueError), (dict(norm_eps=-1.0), RuntimeError),
])
def test_what_it_refuses(kw, err):
    with pytest.raises(err):
        layer(**kw)


def test_sizes_that_the_delta_rule_does_not_take():
    with pytest.raises((ValueError, RuntimeError)):
        DeltaLayer(matrix(2 * 96 + 32), matrix(32), matrix(2), matrix(512, 32), torch.zeros((224, 4)), torch.ones(1),
                   torch.zeros(1), torch.ones(32), 1, 1, 96, 32, 1)
