"""A decode step of several requests at once, around the projections that they
share: the residual norm, a projection with each request's low-rank adapter, the
4-bit head, and the logits under each request's penalties, biases and grammar.

    python examples/decode_requests.py            # 6 requests, 8 steps, synthetic weights

Everything of a step runs on one stream without a synchronisation; the chosen
tokens are appended to the requests' histories on the GPU.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import row_gemv_decode_amd as sk  # noqa: E402


class Step:
    """One layer and the head for a batch of `requests` requests.  Adapter i belongs to
    the requests whose entry of `adapters` is i (negative: none)."""

    def __init__(self, requests, d=1024, vocab=32000, rank=16, pool=4, room=64, group=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, sd):
            return (torch.randn(shape, generator=gen, device=device) * sd).to(torch.bfloat16)

        self.embed = normal(vocab, d, sd=1.0)
        self.norm1, self.norm2 = normal(d, sd=0.1) + 1, normal(d, sd=0.1) + 1
        self.proj = normal(d, d, sd=d ** -0.5)
        self.pool = sk.Adapters(normal(pool, rank, d, sd=d ** -0.5), normal(pool, d, rank, sd=rank ** -0.5),
                                scaling=torch.linspace(0.5, 1.5, pool, device=device))
        codes = torch.randint(0, 256, (vocab, d // 2), generator=gen, device=device, dtype=torch.uint8)
        scales = (torch.rand((vocab, d // group), generator=gen, device=device) + 0.5) * (d ** -0.5 / 4.6)
        self.head = sk.W4(codes, scales.to(torch.bfloat16))
        # what the rules read, filled in place from step to step
        i32 = dict(dtype=torch.int32, device=device)
        self.adapters = torch.full((requests,), -1, **i32)
        self.history = torch.zeros((requests, room), dtype=torch.int64, device=device)
        self.lengths, self.prompts = torch.zeros(requests, **i32), torch.zeros(requests, **i32)
        self.repetition = torch.ones(requests, device=device)
        self.presence = torch.zeros(requests, device=device)
        self.frequency = torch.zeros(requests, device=device)
        self.mask = torch.full((requests, (vocab + 31) // 32), -1, **i32)
        self.mask_rows = torch.full((requests,), -1, **i32)
        self.rules = sk.LogitRules(requests, vocab, history=self.history, lengths=self.lengths, prompt_lengths=self.prompts,
                                   repetition=self.repetition, frequency=self.frequency, presence=self.presence, mask=self.mask,
                                   mask_rows=self.mask_rows)
        self.vocab, self.d = vocab, d

    def start(self, prompts):
        """The requests' prompts, lists of token ids, of at least one token and no more than
        the histories' room."""
        room = self.history.shape[1]
        if len(prompts) != len(self.lengths) or any(not 1 <= len(p) <= room or min(p) < 0 or max(p) >= self.vocab for p in prompts):
            raise ValueError(f"takes {len(self.lengths)} prompts of 1 to {room} tokens below {self.vocab}")
        for i, p in enumerate(prompts):
            self.history[i, :len(p)] = torch.tensor(p, dtype=torch.int64, device=self.history.device)
            self.lengths[i] = self.prompts[i] = len(p)

    def allow(self, request, tokens):
        """Only these tokens for a request from now on."""
        words = torch.zeros((self.mask.shape[1] * 32,), dtype=torch.int64)
        words[torch.tensor(tokens)] = 1
        packed = (words.view(-1, 32) << torch.arange(32)).sum(1)
        self.mask[request] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
        self.mask_rows[request] = request

    def logits(self):
        """Each request's next logits, before and after its rules."""
        last = self.history.gather(1, (self.lengths.long() - 1).unsqueeze(1)).squeeze(1)
        residual = self.embed[last]
        y = sk.rms_norm(residual, self.norm1).out
        out = sk.mm(y, self.proj, out_dtype=torch.bfloat16)
        sk.add_adapters(y, self.pool, self.adapters, out, out=out)
        y = sk.rms_norm(out, self.norm2, residual=residual, residual_out=residual).out
        raw = sk.mm_w4(y, self.head)
        return raw, sk.adjust_logits(raw, self.rules)

    def step(self):
        """The most likely tokens and their log probabilities, appended to the
        histories.  A history whose room is used up stays as it is, also where a captured
        step is replayed."""
        _, logits = self.logits()
        tokens = logits.argmax(1)
        scores = sk.token_logprobs(logits, tokens)
        room = self.history.shape[1]
        place = self.lengths.long().clamp(max=room - 1).unsqueeze(1)
        free = self.lengths < room
        self.history.scatter_(1, place, torch.where(free, tokens, self.history.gather(1, place).squeeze(1)).unsqueeze(1))
        self.lengths += free
        return tokens, scores.logprob


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    prompts = [[17 * i + 1, 5, 9] for i in range(a.requests)]
    s = Step(a.requests, room=max(len(p) for p in prompts) + a.steps)
    s.start(prompts)
    s.adapters.copy_(torch.arange(a.requests, device="cuda") % 5 - 1)
    s.repetition.fill_(1.2)
    s.presence.fill_(0.3)
    s.allow(0, list(range(100, 120)))
    for _ in range(a.steps):
        s.step()
    for i in range(a.requests):
        print(f"request {i} (adapter {int(s.adapters[i])}): {s.history[i, :int(s.lengths[i])].tolist()}")


if __name__ == "__main__":
    main()
