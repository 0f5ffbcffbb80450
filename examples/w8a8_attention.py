#!/usr/bin/env python3
"""A W8A8 attention block served from the 8-bit paged cache.

    python examples/w8a8_attention.py [--seqs 4] [--prompt 300] [--steps 32]

One block of a decoder as a serving loop runs it, every product and the cache in
8 bits: smooth + quantize the hidden states, the fused QKV projection, rotation
and append to the pages, attention, and the output projection of its result.
Ragged prompts go first, in one call; then every sequence gets one token per
step, the step captured once as a HIP graph and replayed while the device-side
lengths grow.  Weights and hidden states are random.  Prints the time of both
and how far the block is from the same block in fp32 with an unquantized cache.
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

PAGE = 64
SMOOTH_ALPHA = 0.85


class Linear:
    """SmoothQuant W8A8 layer: fp16 in, fp16 out."""

    def __init__(self, torch, qlin, W, calib, max_tokens):
        self.q, self.N, self.K = qlin, *W.shape
        s, inv = qlin.sq_compute_smoothing(qlin.sq_act_absmax(calib), W, SMOOTH_ALPHA)
        Wq, ws = qlin.sq_pack_weight(W, s)
        self.inv, self.Wq, self.ws = (torch.from_numpy(a).cuda() for a in (inv, Wq, ws))
        self.Xq = torch.empty((max_tokens, self.K), dtype=torch.int8, device="cuda")
        self.xs = torch.empty(max_tokens, dtype=torch.float32, device="cuda")
        # the workspace grows with the number of tokens only up to a point: the largest of a few sizes
        need = max(qlin.sq_int8_gemm_workspace_bytes(m, self.N, self.K) for m in (max_tokens, 64, 256, 1024))
        self.workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")

    def __call__(self, X, out):
        T = X.shape[0]
        self.q.sq_smooth_quant_act(X, self.inv, T, self.K, self.Xq[:T], self.xs[:T])
        self.q.sq_int8_gemm(self.Xq[:T], self.xs[:T], self.Wq, self.ws, T, self.N, self.K, out, workspace=self.workspace)


class Block:
    def __init__(self, hidden=1024, q_heads=8, kv_heads=2, dim=128, seqs=4, max_len=1024, max_tokens=4096, seed=0):
        import torch

        from quantized_linear_layers_packed_amd import qlin
        self.torch, self.qlin = torch, qlin
        self.hidden, self.q_heads, self.kv_heads, self.dim, self.seqs = hidden, q_heads, kv_heads, dim, seqs
        r = np.random.default_rng(seed)
        width = (q_heads + 2 * kv_heads) * dim
        self.W_qkv = (r.standard_normal((width, hidden)) / math.sqrt(hidden)).astype(np.float32)
        self.W_out = (r.standard_normal((hidden, q_heads * dim)) / math.sqrt(q_heads * dim)).astype(np.float32)
        calib = r.standard_normal((64, hidden)).astype(np.float16)
        self.qkv_layer = Linear(torch, qlin, self.W_qkv, calib, max_tokens)
        calib = (0.3 * r.standard_normal((64, q_heads * dim))).astype(np.float16)
        self.out_layer = Linear(torch, qlin, self.W_out, calib, max_tokens)
        # the pool, and pages dealt out to the sequences in no particular order
        per_seq = -(-max_len // PAGE)
        pages = seqs * per_seq
        self.k = torch.empty((pages, kv_heads, PAGE, dim), dtype=torch.int8, device="cuda")
        self.v = torch.empty((pages, kv_heads, dim, PAGE), dtype=torch.int8, device="cuda")
        self.scales = torch.empty((pages, kv_heads, 2), dtype=torch.float32, device="cuda")
        self.cache = qlin.Kv8Cache(self.k, self.v, self.scales)
        self.table = torch.from_numpy(r.permutation(pages).astype(np.int32).reshape(seqs, per_seq)).cuda()
        self.kv_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        angle = np.arange(max_len)[:, None] * 10000.0 ** (-2.0 * np.arange(dim // 2) / dim)
        self.cos, self.sin = (torch.from_numpy(f(angle).astype(np.float32)).cuda() for f in (np.cos, np.sin))
        self.max_len = max_len

    def plan(self, new, max_kv):
        """What stays the same between steps of the same shape: the batch, its buffers and the workspace."""
        torch, qlin = self.torch, self.qlin
        T = sum(new)
        half = dict(dtype=torch.float16, device="cuda")
        offsets = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32, device="cuda")
        batch = qlin.Kv8Batch(offsets, self.kv_lens, self.table, T, max(new), max_kv)
        need = qlin.qlin_kv8_attention_workspace_bytes(self.cache, batch, self.q_heads)
        return dict(T=T, batch=batch, X=torch.empty((T, self.hidden), **half),
                    qkv=torch.empty((T, self.q_heads + 2 * self.kv_heads, self.dim), **half),
                    q=torch.empty((T, self.q_heads, self.dim), **half), y=torch.empty((T, self.q_heads, self.dim), **half),
                    out=torch.empty((T, self.hidden), **half),
                    workspace=torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None)

    def forward(self, p):
        """p["X"] -> p["out"]; kv_lens already counts the new tokens."""
        qlin, H, G = self.qlin, self.kv_heads, self.q_heads
        self.qkv_layer(p["X"], p["qkv"])
        qkv = p["qkv"]
        qlin.qlin_kv8_append(self.cache, p["batch"], qkv[:, :G], qkv[:, G:G + H], qkv[:, G + H:], qlin.QLIN_F16, G,
                             self.cos, self.sin, self.dim, qlin.QLIN_ROPE_HALF, p["q"])
        qlin.qlin_kv8_attention(self.cache, p["batch"], p["q"], qlin.QLIN_F16, G, 1.0 / math.sqrt(self.dim), 0, 0, p["y"],
                                p["workspace"])
        self.out_layer(p["y"].view(p["T"], -1), p["out"])

    def plain(self, X):
        """The same block in fp32 for one sequence X [tokens][hidden] from its start, nothing quantized."""
        torch, G, H, D = self.torch, self.q_heads, self.kv_heads, self.dim
        T = X.shape[0]
        x = X.float() @ torch.from_numpy(self.W_qkv).cuda().T
        x = x.view(T, G + 2 * H, D)
        a, b = x[:, :G + H, :D // 2], x[:, :G + H, D // 2:]
        c, s = self.cos[:T, None], self.sin[:T, None]
        qk = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
        q, k, v = qk[:, :G], qk[:, G:], x[:, G + H:]
        k, v = (t.repeat_interleave(G // H, dim=1).transpose(0, 1).contiguous() for t in (k, v))
        w = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) / math.sqrt(D)
        w = torch.softmax(w.masked_fill(torch.ones(T, T, device="cuda", dtype=torch.bool).triu(1), -math.inf), dim=-1)
        y = torch.matmul(w, v).transpose(0, 1).reshape(T, G * D)
        return y @ torch.from_numpy(self.W_out).cuda().T


def serve(seqs=4, prompt=300, steps=32, seed=0):
    """Runs prompts and decode steps; returns (relative difference from the fp32 block, ms of the prompts, us per step)."""
    import torch
    r = np.random.default_rng(seed + 1)
    new = [max(1, prompt - 37 * b) for b in range(seqs)]
    block = Block(seqs=seqs, max_len=prompt + steps, max_tokens=max(sum(new), seqs), seed=seed)
    X = [torch.from_numpy(r.standard_normal((n + steps, block.hidden)).astype(np.float16)).cuda() for n in new]
    got = [[] for _ in new]

    def keep(out, counts):
        at = 0
        for b, n in enumerate(counts):
            got[b].append(out[at:at + n].clone())
            at += n

    p = block.plan(new, max(new))
    p["X"].copy_(torch.cat([x[:n] for x, n in zip(X, new)]))
    block.kv_lens.copy_(torch.tensor(new, dtype=torch.int32))
    block.forward(p)                                       # loads the kernels
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    block.forward(p)                                       # appending the same tokens again changes nothing
    torch.cuda.synchronize()
    prompt_ms = (time.perf_counter() - t0) * 1e3
    keep(p["out"], new)

    # One token per sequence and step, as a graph: the lengths grow on the device.
    p = block.plan([1] * seqs, block.max_len)
    lens = block.kv_lens.clone()
    block.kv_lens.add_(1)
    p["X"].zero_()
    block.forward(p)                                       # kernels loaded and buffers made before the capture
    torch.cuda.synchronize()
    block.kv_lens.copy_(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.kv_lens.add_(1)
        block.forward(p)
    block.kv_lens.copy_(lens)                              # the trial token's slot is overwritten by the first step
    total = 0.0
    for i in range(steps):
        p["X"].copy_(torch.stack([x[n + i] for x, n in zip(X, new)]))
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        total += time.perf_counter() - t0
        keep(p["out"], [1] * seqs)
    off, size = 0.0, 0.0
    for b, x in enumerate(X):
        ref = block.plain(x)
        off += float((torch.cat(got[b]).float() - ref).square().sum())
        size += float(ref.square().sum())
    return math.sqrt(off / size), prompt_ms, total / max(steps, 1) * 1e6


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    diff, prompt_ms, step_us = serve(a.seqs, a.prompt, a.steps)
    print(f"{a.seqs} sequences: prompts {prompt_ms:.2f} ms, one token each {step_us:.0f} us, "
          f"relative difference from the fp32 block {diff:.4f}")


if __name__ == "__main__":
    main()
