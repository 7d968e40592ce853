"""One decode window through the library's window operators: a mixture-of-experts
layer, the 4-bit output head, and the log probabilities of the tokens a
speculative decoder has drafted.

    python examples/decode_window.py            # 6 rows on synthetic weights

The three run one after another on one stream, without a synchronisation
between them; the accepted prefix is the only thing that is read back.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import row_gemv_decode_amd as sk  # noqa: E402


def grouped_w4(shape, group, gen, dtype=torch.bfloat16, sd=0.02):
    """A synthetic 4-bit weight [..., k] with random codes and zero points 7 .. 9,
    its values about N(0, sd)."""
    *rows, k = shape
    codes = torch.randint(0, 256, (*rows, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((*rows, k // group), generator=gen, device="cuda") + 0.5) * (sd / 4.6)
    zeros = torch.randint(7, 10, (*rows, k // group), generator=gen, device="cuda", dtype=torch.uint8)
    return sk.W4(codes, scales.to(dtype), zeros)


class Window:
    """The last layer's experts, the head, and the scoring of a window."""

    def __init__(self, experts=64, topk=6, d=1024, inter=512, shared=512, vocab=32000, group=64, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def half(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * 0.03).to(torch.bfloat16)

        self.layer = sk.MoELayer(half(experts, d), grouped_w4((experts, 2 * inter, d), group, gen),
                                 grouped_w4((experts, d, inter), group, gen), topk=topk,
                                 shared13=grouped_w4((2 * shared, d), group, gen),
                                 shared2=grouped_w4((d, shared), group, gen), shared_gate=half(d))
        self.head = grouped_w4((vocab, d), group, gen)

    def score(self, x, drafted, alternatives=5):
        """x [m][d], m <= 16 rows; drafted [m] token ids: the rows' logits and the
        drafted tokens' log probabilities, ranks and top alternatives."""
        y = x + self.layer(x)
        logits = sk.mm_w4(y, self.head)
        return logits, sk.token_logprobs(logits, drafted, topk=alternatives)


def accepted(scores):
    """How many drafted tokens from the first on are the most likely ones."""
    return int((scores.rank == 1).to(torch.int32).cumprod(0).sum())


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rows", type=int, default=6)
    a = ap.parse_args()
    w = Window()
    x = torch.randn((a.rows, w.layer.d), device="cuda").to(torch.bfloat16)
    logits, _ = w.score(x, torch.zeros(a.rows, dtype=torch.int64, device="cuda"))
    drafted = logits.argmax(1)
    drafted[a.rows // 2] += 1  # a draft that goes wrong half way (the id past the best one)
    drafted %= logits.shape[1]
    _, s = w.score(x, drafted)
    for i in range(a.rows):
        alt = ", ".join(f"{t} ({p:.2f})" for t, p in zip(s.top_ids[i].tolist(), s.top_logprobs[i].tolist()))
        print(f"row {i}: token {int(drafted[i])} log p {float(s.logprob[i]):.3f} rank {int(s.rank[i])} "
              f"entropy {float(s.entropy[i]):.3f} nats; top: {alt}")
    print(f"accepted {accepted(s)} of {a.rows}")


if __name__ == "__main__":
    main()
