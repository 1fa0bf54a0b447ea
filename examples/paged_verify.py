"""Tree-verify steps over a paged 4-bit key/value cache, on random weights.

Two requests with prompts of different lengths, packed one behind the other, share a
pool of pages: their queries and keys are rotated, their keys and values cached. Each
step scores a draft tree per request, the second with a low-rank adapter of the first
product: pages are reserved, the layer's products and attention run over the 4-bit
cache, the deepest accepted path is answered with its log probabilities, its rows are
committed and the pages of the rest given back.

    python examples/paged_verify.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_w12_gb300 import synthetic as S  # noqa: E402
from speculative_decoding_verification_w12_gb300 import w12  # noqa: E402
from speculative_decoding_verification_w12_gb300.engine import PagedVerifyStep  # noqa: E402


def weights(N, K, seed):
    bits = torch.from_numpy(S.weights_bf16(N, K, seed=seed).view("int16")).cuda()
    return w12.pack(bits.view(torch.bfloat16))


def adapters(N, K, n=4, rank=16):
    g = torch.Generator(device="cuda").manual_seed(9)
    A, B = (torch.randn(s, generator=g, device="cuda") * 0.02 for s in ((n, rank, K), (n, N, rank)))
    return w12.LoRA(A.bfloat16(), B.bfloat16(), torch.ones(n, device="cuda"))


def main(steps=3, B=2, T=16, hidden=512, Hq=10, Hkv=2, d=64, vocab=4096):
    step = PagedVerifyStep(weights((Hq + 2 * Hkv) * d, hidden, 1), weights(hidden, Hq * d, 2), weights(vocab, hidden, 3),
                           B, T, Hq, Hkv, d, n_pages=64, page_size=16, max_len=512, top_k=3,
                           rope=w12.Rope.create(d, 512, q_norm=torch.ones(d, device="cuda"), k_norm=torch.ones(d, device="cuda")),
                           adapters={"qkv": adapters((Hq + 2 * Hkv) * d, hidden)})
    g = torch.Generator(device="cuda").manual_seed(0)
    cu = torch.tensor([0, 37, 187], dtype=torch.int32, device="cuda")
    step.prompt(*(torch.randn((187, H, d), generator=g, device="cuda") for H in (Hq, Hkv, Hkv)), cu)
    mine = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    parents = torch.tensor([list(range(-1, T - 1)), [-1] + [(i - 1) // 2 for i in range(1, T)]], dtype=torch.int32,
                           device="cuda")  # a chain, and a binary tree
    for n in range(steps):
        X = torch.randn((B * T, hidden), generator=g, device="cuda").bfloat16()
        draft = torch.randint(0, vocab, (B, T), generator=g, device="cuda", dtype=torch.int32)
        r = step.run(X, parents, draft, adapter=mine)
        if int(step.status.item()):
            raise w12.W12Error(int(step.status.item()), "verify step")
        for b in range(B):
            k = int(r["accept_len"][b]) + 1
            print(f"step {n} request {b}: tokens {r['tokens'][b, :k].tolist()}, logprobs "
                  f"{[round(x, 2) for x in r['logprob'][b, :k].tolist()]}, entropy {float(r['entropy'][b, 0]):.2f}, "
                  f"length {int(step.length[b])}, pages {int(step.pages.used[b])}")


if __name__ == "__main__":
    main()
