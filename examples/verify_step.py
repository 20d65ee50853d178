"""Speculative decoding of requests that each have an adapter and a temperature, on 4-bit weights.

The model is one 4-bit product from a token's embedding to the logits of the next one. Drafts come from it without the
adapters, then one step verifies all of them:

    product (mnb_gemm) -> each row's adapter (mnb_lora, in place) -> probabilities (mnb_softmax) ->
    accepted tokens and the next one (mnb_verify)

Run as ``python examples/verify_step.py [--batch B] [--drafts N] [--steps S]``; it prints how many drafted tokens a step
accepts and the time of the verifying part, eager and as a captured CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gemm_mnb_gemv_gb300 as mnb  # noqa: E402
from examples.decode_layer import Weight  # noqa: E402


class Model:
    def __init__(self, vocab, hidden, adapters, rank, device="cuda"):
        self.V = vocab
        rand = lambda *shape: torch.randn(shape, device=device, dtype=torch.float16)  # noqa: E731
        self.embedding = rand(vocab, hidden)
        self.head = Weight("verify_head", hidden, vocab, 32, device)
        ranks = torch.randint(rank // 2, rank + 1, (adapters,), device=device, dtype=torch.int32)
        scales = torch.full((adapters,), 0.5, device=device)
        self.pool = mnb.MnbLoraPool(rand(adapters, rank, hidden) / hidden ** 0.5, rand(adapters, vocab, rank) / rank ** 0.5,
                                    ranks, scales)

    def probabilities(self, tokens, temperature, adapter=None):
        x = self.embedding[tokens]
        y = self.head(x)
        if adapter is not None:
            mnb.mnb_lora(x, self.pool, adapter, base=y, out=y)
        return mnb.mnb_softmax(y, temperature)


def run(batch=16, drafts=4, steps=20, vocab=32000, hidden=2048, adapters=8, rank=16, device="cuda"):
    """(accepted tokens a step and sequence, ms of an eager verification, ms of a captured one)"""
    torch.manual_seed(1)
    model = Model(vocab, hidden, adapters, rank, device)
    n = drafts
    per_row = lambda v: v.repeat_interleave(n + 1)  # noqa: E731
    adapter = torch.randint(-1, adapters, (batch,), device=device, dtype=torch.int32)
    warmth = torch.linspace(0.0, 1.2, batch, device=device)
    rows_adapter, rows_warmth = per_row(adapter), per_row(warmth)
    start = torch.arange(0, batch * n + 1, n, dtype=torch.int32, device=device)
    last = torch.randint(0, vocab, (batch,), device=device)

    def verify(inputs, draft, drafted, u, v):
        p = model.probabilities(inputs, rows_warmth, rows_adapter)
        return mnb.mnb_verify(p, draft, drafted, start, u, v)

    taken, times = 0, []
    for _ in range(steps):
        row, draft, drafted = last, [], []
        for _ in range(n):
            q = model.probabilities(row, warmth)
            row = torch.multinomial(q, 1)[:, 0]
            draft.append(q), drafted.append(row)
        draft, drafted = torch.stack(draft, 1).view(-1, vocab), torch.stack(drafted, 1)
        inputs = torch.cat([last[:, None], drafted], 1).view(-1)
        case = (inputs, draft, drafted.view(-1).int(), torch.rand(batch * n, device=device), torch.rand(batch, device=device))
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        tokens, accepted = verify(*case)
        b.record()
        last = tokens.view(batch, n + 1).gather(1, accepted.long()[:, None])[:, 0].long()
        taken += int(accepted.sum())
        times.append(a.elapsed_time(b))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = verify(*case)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(20):
        graph.replay()
    b.record()
    b.synchronize()
    if not (torch.equal(again[0], tokens) and torch.equal(again[1], accepted)):
        raise AssertionError("the captured step differs from the eager one")
    mnb.mnb_check_device_status()
    return taken / steps / batch, sorted(times)[len(times) // 2], a.elapsed_time(b) / 20


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--batch", type=int, default=16)
    parser.add_argument("--drafts", type=int, default=4)
    parser.add_argument("--steps", type=int, default=20)
    args = parser.parse_args()
    accepted, eager, captured = run(args.batch, args.drafts, args.steps)
    print(f"{args.batch} sequences, {args.drafts} drafted tokens each: {accepted:.2f} accepted; verification {eager * 1e3:.1f} us, "
          f"captured {captured * 1e3:.1f} us")
