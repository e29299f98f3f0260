"""Prompts, then decode steps, over a 4-bit key/value cache.

What a serving loop does with the mx_kv_* calls: every sequence has pages of
one pool, new keys and values are quantised into their slots as they come out
of the projection, and attention reads the codes.  Prompts are attended to in
one call over ragged queries, then each step writes one token per sequence and
attends again; the step is captured into a CUDA graph and replayed with new
inputs and lengths.

    python examples/kv_cache_step.py

Prints how far the outputs are from attention over the very values that the
cache holds, and over the unquantised keys and values (random ones, which are
harder on 4 bits than a model's).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tensor_scaling_cast_gb300 import fp8q as F  # noqa: E402

Q_HEADS, KV_HEADS, HEAD_DIM, PAGE = 16, 4, 128, 16


def reference(q, k, v, first):
    """softmax(q k^T / sqrt(D)) v in fp32 for queries at positions first, first + 1, .."""
    group = q.shape[1] // k.shape[1]
    k, v = (x.float().repeat_interleave(group, 1) for x in (k, v))
    s = torch.einsum("qhd,khd->hqk", q.float(), k) * q.shape[2] ** -0.5
    pos = first + torch.arange(q.shape[0], device=q.device)
    s = s.masked_fill(torch.arange(k.shape[0], device=q.device) > pos[:, None], -torch.inf)
    return torch.einsum("hqk,khd->qhd", s.softmax(-1), v)


def off(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


def main(prompts=(900, 33, 2500, 128), steps=8, seed=0, quiet=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    batch, longest = len(prompts), max(prompts) + steps
    per = -(-longest // PAGE)
    cache = F.MXKVCache.allocate(batch * per, PAGE, KV_HEADS, HEAD_DIM)
    table = torch.randperm(batch * per, generator=gen, device="cuda").int().view(batch, per)
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    kept = [[] for _ in prompts]                     # the unquantised keys and values, for the comparison

    def project(tokens):
        """One projection's output: queries, keys and values of every token in one row."""
        x = torch.randn(tokens, Q_HEADS + 2 * KV_HEADS, HEAD_DIM, generator=gen, device="cuda").bfloat16()
        return x[:, :Q_HEADS], x[:, Q_HEADS:Q_HEADS + KV_HEADS], x[:, Q_HEADS + KV_HEADS:]

    def slots_of(seq, first, n):
        t = torch.arange(first, first + n, device="cuda")
        return table[seq, t // PAGE].long() * PAGE + t % PAGE

    # prompts: one write, one attention call over ragged queries
    q, k, v = project(sum(prompts))
    cu = torch.tensor([0] + list(prompts), device="cuda").cumsum(0).int()
    slots = torch.cat([slots_of(b, 0, n) for b, n in enumerate(prompts)])
    F.mx_kv_write(cache, k, v, slots, rule=F.MX_CEIL)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    workspace = F.mx_kv_attention_workspace(cache, q, table, max_q=max(prompts))
    F.mx_kv_attention(cache, q, out, table, lens, cu_q=cu, max_q=max(prompts), workspace=workspace)
    for b in range(batch):
        kept[b] += [(k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])]

    # steps: one token per sequence, the same two calls in a graph
    step_q, step_k, step_v = (torch.zeros(batch, h, HEAD_DIM, dtype=torch.bfloat16, device="cuda")
                              for h in (Q_HEADS, KV_HEADS, KV_HEADS))
    step_slots = torch.full((batch,), -1, device="cuda")
    step_out = torch.empty_like(step_q)
    step_ws = F.mx_kv_attention_workspace(cache, step_q, table, max_q=1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.mx_kv_write(cache, step_k, step_v, step_slots, rule=F.MX_CEIL)
        F.mx_kv_attention(cache, step_q, step_out, table, lens, workspace=step_ws)
    made = []
    for b, n in enumerate(prompts):
        made.append((out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], b, 0, n))
    for _ in range(steps):
        q, k, v = project(batch)
        step_q.copy_(q), step_k.copy_(k), step_v.copy_(v)
        at = lens.long()
        step_slots.copy_(table[torch.arange(batch, device="cuda"), at // PAGE].long() * PAGE + at % PAGE)
        lens += 1
        graph.replay()
        for b in range(batch):
            kept[b].append((k[b:b + 1], v[b:b + 1]))
            made.append((step_out[b:b + 1].clone(), q[b:b + 1], b, int(at[b]), int(at[b]) + 1))

    worst = [0.0, 0.0]
    for got, q, b, first, n in made:
        k_c, v_c = (torch.empty(n, KV_HEADS, HEAD_DIM, device="cuda") for _ in range(2))
        F.mx_kv_read(cache, slots_of(b, 0, n), k_c, v_c)
        plain = [torch.cat(x)[:n] for x in zip(*kept[b])]
        worst[0] = max(worst[0], off(got, reference(q, k_c, v_c, first)))
        worst[1] = max(worst[1], off(got, reference(q, *plain, first)))
    if not quiet:
        print(f"{batch} sequences, prompts {tuple(prompts)}, {steps} steps: largest relative difference "
              f"{worst[0]:.2e} over the cached values, {worst[1]:.2e} over the unquantised ones")
    return worst


if __name__ == "__main__":
    main()
