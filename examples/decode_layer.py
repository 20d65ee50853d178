"""The attention half of a decoder layer on 4-bit weights and a 4-bit key/value cache.

Prefill of a batch of prompts, then decode steps from one captured CUDA graph:

    qkv product (mnb_gemm) -> rotate, quantise and append (mnb_kv4_append) -> attention over the cache
    (mnb_kv4_attention) -> output product (mnb_gemm)

Run as ``python examples/decode_layer.py [--batch B] [--prompt P] [--steps N]``; it prints the time of
the prefill and of a decode step, and checks the last step's attention against fp32 torch on the
values that the cache holds (mnb_kv4_read).
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
import mnb_synth as syn  # noqa: E402


class Weight:
    """One MatMulNBits weight on the device, with its tensor-core copy for more than 16 rows."""

    def __init__(self, name, K, N, block_size, device):
        w = syn.make_weight(syn.custom(name, 1, K, N, block_size, scale_lo=0.2 / K ** 0.5, scale_hi=0.4 / K ** 0.5))
        self.K, self.N, self.block_size = K, N, block_size
        self.parts = tuple(torch.from_numpy(a).to(device) for a in (w.packed, w.scales, w.zero_points))
        self.repacked = mnb.mnb_repack(self.parts[0], K, N, block_size)

    def __call__(self, x):
        return mnb.mnb_gemm(x, *self.parts, self.K, self.N, self.block_size, repacked=self.repacked)


class AttentionLayer:
    def __init__(self, batch, max_tokens, q_heads=32, kv_heads=8, head_dim=128, hidden=4096, group_size=64, page_size=64,
                 device="cuda"):
        self.B, self.Hq, self.Hk, self.D, self.page_size = batch, q_heads, kv_heads, head_dim, page_size
        self.qkv = Weight("layer_qkv", hidden, (q_heads + 2 * kv_heads) * head_dim, 32, device)
        self.out = Weight("layer_out", q_heads * head_dim, hidden, 32, device)
        pages = -(-max_tokens // page_size)
        self.cache = mnb.mnb_kv4_cache_alloc(batch * pages, page_size, kv_heads, head_dim, group_size, device)
        # pages are dealt out to the sequences in turn
        self.table = torch.arange(batch * pages, dtype=torch.int32, device=device).view(pages, batch).t().contiguous()
        inv = 10000.0 ** (-torch.arange(head_dim // 2, dtype=torch.float64) / (head_dim // 2))
        angle = torch.arange(max_tokens, dtype=torch.float64)[:, None] * inv
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.scale = head_dim ** -0.5

    def forward(self, x, q_start, positions, seq):
        """x ``[T, hidden]``: new tokens of the sequences ``seq`` at ``positions``; kv_len already counts them."""
        T, D = x.shape[0], self.D
        y = self.qkv(x)
        q, k, v = (t.view(T, -1, D) for t in y.split([self.Hq * D, self.Hk * D, self.Hk * D], dim=1))
        slots = self.table[seq, (positions // self.page_size).long()].long() * self.page_size + positions % self.page_size
        q = mnb.mnb_kv4_append(self.cache, k, v, slots, q=q, positions=positions, cos=self.cos, sin=self.sin)
        o = mnb.mnb_kv4_attention(q, self.cache, q_start, self.kv_len, self.table, self.scale)
        return self.out(o.view(T, self.Hq * D)), q, o

    def prefill(self, x, lengths):
        """x: the prompts' tokens one after the other; lengths: tokens of each prompt (a list)."""
        dev = x.device
        n = torch.tensor(lengths, dtype=torch.int64, device=dev)
        start = torch.zeros(self.B + 1, dtype=torch.int32, device=dev)
        start[1:] = n.cumsum(0)
        seq = torch.repeat_interleave(torch.arange(self.B, device=dev), n)
        positions = (torch.arange(x.shape[0], device=dev) - start[:-1].long()[seq]).int()
        self.kv_len.copy_(n)
        return self.forward(x, start, positions, seq)

    def capture_step(self, x):
        """A graph of one decode step on the buffer x ``[B, hidden]``; returns it with the step's (y, q, o)."""
        start = torch.arange(self.B + 1, dtype=torch.int32, device=x.device)
        seq = torch.arange(self.B, device=x.device)

        def step():
            positions = self.kv_len.clone()
            self.kv_len += 1
            return self.forward(x, start, positions, seq)

        kept = self.kv_len.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        self.kv_len.copy_(kept)  # the warm-up's token is written again by the first replay
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outputs = step()
        return graph, outputs


def reference_attention(layer, q):
    """fp32 attention of one token a sequence over the values that the cache holds."""
    out = torch.empty_like(q)
    for b, n in enumerate(layer.kv_len.tolist()):
        j = torch.arange(n, device=q.device)
        slots = layer.table[b, j // layer.page_size].long() * layer.page_size + j % layer.page_size
        k, v = mnb.mnb_kv4_read(layer.cache, slots, dtype=torch.float32)
        qb = q[b].float().view(layer.Hk, -1, layer.D)
        p = torch.einsum("hgd,jhd->hgj", qb, k).mul(layer.scale).softmax(-1)
        out[b] = torch.einsum("hgj,jhd->hgd", p, v).reshape(layer.Hq, layer.D).to(q.dtype)
    return out


def run(batch=4, prompt=512, steps=32, **layer_args):
    """Returns (prefill us, decode step us, relative error of the last step's attention)."""
    dev = torch.device("cuda")
    lengths = [max(1, prompt - 37 * b) for b in range(batch)]
    layer = AttentionLayer(batch, prompt + steps + 1, device=dev, **layer_args)
    hidden = layer.qkv.K
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    x = torch.randn(sum(lengths), hidden, generator=gen, device=dev).half()
    layer.prefill(x, lengths)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    t[0].record()
    layer.prefill(x, lengths)
    t[1].record()
    token = torch.randn(batch, hidden, generator=gen, device=dev).half()
    graph, (y, q, o) = layer.capture_step(token)
    t[2].record()
    for _ in range(steps):
        graph.replay()
    t[3].record()
    torch.cuda.synchronize()
    mnb.mnb_check_device_status()
    want = reference_attention(layer, q)
    error = float((o.float() - want.float()).norm() / want.float().norm())
    assert torch.isfinite(y).all()
    return t[0].elapsed_time(t[1]) * 1e3, t[2].elapsed_time(t[3]) * 1e3 / steps, error


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    pre, dec, err = run(a.batch, a.prompt, a.steps)
    print(f"prefill {pre:.1f} us, decode step {dec:.1f} us, attention error against fp32 torch {err:.1e}")
