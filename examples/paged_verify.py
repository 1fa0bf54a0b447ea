"""Tree-verify steps over a paged 4-bit key/value cache, on random weights.

Two requests with prompts of different lengths share a pool of pages. Each step
scores a draft tree per request: pages are reserved, the layer's products and
attention run over the 4-bit cache, the deepest accepted path is answered with its
log probabilities, its rows are committed and the pages of the rest given back.

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


def main(steps=3, B=2, T=16, hidden=512, Hq=10, Hkv=2, d=64, vocab=4096):
    step = PagedVerifyStep(weights((Hq + 2 * Hkv) * d, hidden, 1), weights(hidden, Hq * d, 2), weights(vocab, hidden, 3),
                           B, T, Hq, Hkv, d, n_pages=64, page_size=16, max_len=512, top_k=3)
    g = torch.Generator(device="cuda").manual_seed(0)
    prompt = torch.tensor([37, 150], dtype=torch.int32, device="cuda")
    K, V = (torch.randn((B, 150, Hkv, d), generator=g, device="cuda") for _ in range(2))
    step.prefill(K, V, prompt)
    parents = torch.tensor([list(range(-1, T - 1)), [-1] + [(i - 1) // 2 for i in range(1, T)]], dtype=torch.int32,
                           device="cuda")  # a chain, and a binary tree
    for n in range(steps):
        X = torch.randn((B * T, hidden), generator=g, device="cuda").bfloat16()
        draft = torch.randint(0, vocab, (B, T), generator=g, device="cuda", dtype=torch.int32)
        r = step.run(X, parents, draft)
        if int(step.status.item()):
            raise w12.W12Error(int(step.status.item()), "verify step")
        for b in range(B):
            k = int(r["accept_len"][b]) + 1
            print(f"step {n} request {b}: tokens {r['tokens'][b, :k].tolist()}, logprobs "
                  f"{[round(x, 2) for x in r['logprob'][b, :k].tolist()]}, entropy {float(r['entropy'][b, 0]):.2f}, "
                  f"length {int(step.length[b])}, pages {int(step.pages.used[b])}")


if __name__ == "__main__":
    main()
