"""The attention layer (ternary_hybrid_bit_amd/attention.py) on small packed
matrices: prompts, chunks and single tokens of several sequences through one
cache.

Two tolerances, fixed before the first run:
* between the products, against oracle/attention.py in float64 on the products'
  own outputs: attend_bound, and what the rounding of the rotated q and k to bf16
  (2^-8 of an element each, so 2^-7 of a score's terms, with the second order
  2.1 2^-8 each way) moves the weights by: twice that times the sum of w |v|;
* prompt() against forward(): both within that bound of the same values.
"""
import numpy as np
import pytest

from oracle import attention as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HIDDEN, QH, KVH, D = 512, 8, 2, 64


@pytest.fixture(scope="module")
def mod():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    from ternary_hybrid_bit_amd import attention
    return attention


@pytest.fixture(scope="module")
def mats(mod):
    return mod.packed_layer(11, HIDDEN, QH, KVH, D)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def reference(layer, X, lens):
    """Oracle attention of whole sequences from the layer's own q, k, v products; per element its bound."""
    q, k, v = (host(layer._product(m, X)).reshape(X.shape[0], -1, D) for m in layer.mats[:3])
    v = host(torch.from_numpy(v.reshape(X.shape[0], -1)).to(torch.bfloat16)).reshape(v.shape)
    f, m = A.rope_freqs(D, 1e6)
    out, bound, at = [], [], 0
    for n in lens:
        pos, s = np.arange(n), slice(at, at + n)
        qr, kr = A.rope(q[s], pos, f, m)[0], A.rope(k[s], pos, f, m)[0]
        o, size, most = A.attend(qr, kr, v[s], pos, D ** -0.5)
        moved = 2 * np.expm1(2.1 * 2.0 ** -8 * most)[..., None] * size
        out.append(o)
        bound.append(A.attend_bound(o, size, most, D, n) + moved)
        at += n
    return np.concatenate(out).reshape(X.shape[0], -1), np.concatenate(bound).reshape(X.shape[0], -1)


def test_prompts_chunks_and_tokens(mod, mats):
    lens = [70, 33, 5]
    X = torch.randn((sum(lens), HIDDEN), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    layer = mod.AttentionLayer(*mats, head_dim=D, n_pages=20, max_seqs=3, page_size=16)
    ref, bound = reference(layer, X, lens)
    starts = np.cumsum([0] + lens)
    Q, K, V = (layer._product(m, X) for m in layer.mats[:3])
    got = torch.full((X.shape[0], QH * D), float("nan"), device="cuda")
    done = [0, 0, 0]
    for step in ([40, 20, 0], [1, 12, 1], [28, 1, 1], [1, 0, 3]):       # new tokens of each sequence
        seqs = [i for i in range(3) if step[i]]
        rows = np.concatenate([np.arange(starts[i] + done[i], starts[i] + done[i] + step[i]) for i in seqs])
        r = torch.from_numpy(rows).cuda()
        got[r] = layer.attend(Q[r], K[r], V[r], seqs, [step[i] for i in seqs]).float()
        for i in seqs:
            done[i] += step[i]
    assert done == lens and layer.lens == lens
    assert (np.abs(host(got) - ref) <= bound).all()
    # pages come back, and a new sequence in used pages is not disturbed by what they held
    layer.release(0)
    again = layer.attend(Q[:70], K[:70], V[:70], [0], [70])
    assert (np.abs(host(again) - ref[:70]) <= bound[:70]).all()


@pytest.mark.parametrize("fmt", [0, 1])
def test_forward_and_prompt_run_the_products(mod, mats, fmt):
    """forward() and prompt() are the products around the attention: equal to doing them by hand."""
    lens = [50, 20]
    X = torch.randn((70, HIDDEN), device="cuda", generator=torch.Generator("cuda").manual_seed(4)).to(torch.bfloat16)
    one, two = (mod.AttentionLayer(*mats, head_dim=D, n_pages=12, max_seqs=2, page_size=16, fmt=fmt) for _ in range(2))
    y = one.forward(X, [0, 1], lens)
    Q, K, V = (two._product(m, X) for m in two.mats[:3])
    a = two.attend(Q, K, V, [0, 1], lens)
    assert torch.equal(y, two._product(two.mats[3], a))
    if fmt == 0:
        ref, bound = reference(one, X, lens)
        assert (np.abs(host(a) - ref) <= bound).all()
        q, k = (torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in (Q, K))
        whole = one.prompt(X, lens)
        assert whole.shape == y.shape and torch.isfinite(whole).all()
        # the products of two inputs that are both within the bound of the same values
        assert ((whole - y).norm() / y.norm()).item() <= 2 * np.linalg.norm(bound) / np.linalg.norm(ref) * 2
