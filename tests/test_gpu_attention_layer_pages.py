"""The attention layer when its cache is full, and its prompts without a cache, against the float64 oracle with the
tolerance of test_gpu_attention_layer.py."""
import numpy as np
import pytest

from oracle import attention as A

from test_gpu_attention_layer import D, HIDDEN, host, mats, mod, reference  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def inputs(n, seed):
    return torch.randn((n, HIDDEN), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(torch.bfloat16)


def test_again_after_the_pages_ran_out(mod, mats):  # noqa: F811
    """A call that finds no page, a release and the same call again: the sequences' values and positions are right."""
    lens = [16, 40, 23]
    X = inputs(sum(lens), 6)
    layer = mod.AttentionLayer(*mats, head_dim=D, n_pages=6, max_seqs=4, page_size=16)
    ref, bound = reference(layer, X, lens)
    Q, K, V = (layer._product(m, X) for m in layer.mats[:3])
    layer.attend(Q[:5], K[:5], V[:5], [3], [5])
    with pytest.raises(RuntimeError):
        layer.attend(Q, K, V, [0, 1, 2], lens)
    with pytest.raises(RuntimeError):
        layer.forward(X, [0, 1, 2], lens)
    layer.release(3)
    a, b = lens[0], lens[0] + lens[1]
    first = torch.cat([torch.arange(a - 3), torch.arange(a, b - 1), torch.arange(b, len(X))]).cuda()
    last = torch.tensor([a - 3, a - 2, a - 1, b - 1], device="cuda")
    got = torch.empty((len(X), Q.shape[1]), device="cuda")
    got[first] = layer.attend(Q[first], K[first], V[first], [0, 1, 2], [13, 39, 23]).float()
    got[last] = layer.attend(Q[last], K[last], V[last], [0, 1], [3, 1]).float()
    assert (np.abs(host(got) - ref) <= bound).all()


@pytest.mark.parametrize("lens", [[50, 20], [1], [129, 3, 0, 64]])
def test_prompt_per_element(mod, mats, lens, monkeypatch):  # noqa: F811
    """What prompt() hands to the last product is, per element, the attention of the rotated q and k; the rest of prompt() is that product."""
    X = inputs(sum(lens), 9)
    layer = mod.AttentionLayer(*mats, head_dim=D, n_pages=1, max_seqs=1, page_size=16)
    ref, bound = reference(layer, X, lens)
    product, seen = layer._product, []

    def keep(m, x):
        if m is layer.mats[3]:
            seen.append(x)
        return product(m, x)
    layer._product = keep
    whole = layer.prompt(X, lens)
    got = host(seen[0])
    assert len(seen) == 1 and (np.abs(got - ref) <= bound).all()
    assert torch.equal(whole, product(layer.mats[3], seen[0]))
    if max(lens) > 1:                           # an oracle that does not rotate is told apart
        monkeypatch.setattr(A, "rope_freqs", lambda rot, base: (np.zeros(rot // 2), 1.0))
        still, bound = reference(layer, X, lens)
        assert not (np.abs(got - still) <= bound).all()
