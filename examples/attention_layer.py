"""One attention layer of 8B-shaped packed matrices on a prompt and then token
by token, with what a step takes:

    python examples/attention_layer.py
"""
import os
import sys
import time

import torch   # before libwal, so that the process has one HIP runtime

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ternary_hybrid_bit_amd.attention import AttentionLayer, packed_layer  # noqa: E402


def main():
    mats = packed_layer(7, 4096, 32, 8, 128)
    layer = AttentionLayer(*mats, head_dim=128, n_pages=64, max_seqs=1)
    n = 2048
    X = torch.randn((n, 4096), device="cuda").to(torch.bfloat16)
    whole = layer.prompt(X, [n])
    got = layer.forward(X[:-3], [0], [n - 3])
    tail = torch.cat([layer.forward(X[i:i + 1], [0], [1]) for i in range(n - 3, n)])
    err = (torch.cat([got, tail]) - whole).norm() / whole.norm()
    print(f"prompt of {n} tokens at once against the cache, in a chunk and 3 single tokens: relative difference {err:.2e}")
    for name, f in (("a prompt of 2048 tokens", lambda: layer.prompt(X, [n])),
                    ("a token over 2050 tokens and more", lambda: layer.forward(X[:1], [0], [1]))):
        for _ in range(5):
            f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            f()
        torch.cuda.synchronize()
        print(f"{name}: {(time.perf_counter() - t) / 20 * 1e6:.1f} us a layer")


if __name__ == "__main__":
    main()
