#!/usr/bin/env python3
"""A serving loop over an 8-bit key/value cache: prompts, then one token a request and step.

Every step is three calls on the GPU with no copy to the host: kv_tables gives the step's tokens their places (blocks
from a ring of free ones, ended requests' blocks back to it), kv_store quantizes their keys and values into them,
kv_attention reads the cache.  Queries, keys and values are random here, where a model's projections would be.  The
last step is compared with attention over the keys and values as kv_load gives them back.

Usage: python examples/kv_serving.py [--requests 16] [--steps 20] [--code q8|e4m3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_nq_amd as nq  # noqa: E402

HEADS, Q_HEADS, DIM, BLOCK = 8, 32, 128, 64


def check(cache, q, token_start, lengths, table, out):
    """Largest difference from softmax attention over the loaded blocks, relative to the largest output."""
    worst = 0.0
    for r in range(lengths.numel()):
        n, s0, s1 = int(lengths[r]), int(token_start[r]), int(token_start[r + 1])
        if s0 == s1:
            continue
        k, v = (x.reshape(-1, HEADS, DIM)[:n] for x in nq.kv_load(cache, table[r, : -(-n // BLOCK)].contiguous()))
        for h in range(Q_HEADS):
            score = q[s0:s1, h].float() @ k[:, h * HEADS // Q_HEADS].T.contiguous() * DIM ** -0.5
            at = torch.arange(n - (s1 - s0), n, device=q.device)[:, None]
            score = score.masked_fill(torch.arange(n, device=q.device)[None] > at, float("-inf"))
            ref = torch.softmax(score, 1) @ v[:, h * HEADS // Q_HEADS]
            worst = max(worst, float((out[s0:s1, h].float() - ref).abs().max() / ref.abs().max()))
    return worst


def main(requests=16, steps=20, code="q8", prompt=700, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    longest = prompt + steps
    width = -(-longest // BLOCK)
    blocks = requests * width
    cache = nq.KvCache.empty(blocks, HEADS, BLOCK, DIM, code)
    table = torch.full((requests, width), -1, **i32)
    ring = torch.arange(blocks, **i32)
    state = torch.tensor([0, blocks], **i32)
    lengths = torch.zeros(requests, **i32)
    # first the prompts; then one token each, and every fifth step a request ends
    added = torch.randint(1, prompt + 1, (requests,), generator=gen, **i32)
    tokens, most = requests * prompt, prompt
    problems = torch.zeros(1, **i32)
    for i in range(steps):
        step = nq.kv_tables(lengths, added, table, ring, state, BLOCK, tokens)
        q, k, v = new(tokens, Q_HEADS, DIM), new(tokens, HEADS, DIM), new(tokens, HEADS, DIM)
        bad = nq.kv_store(cache, k, v, step.slots, step.token_start)
        out = nq.kv_attention(cache, q, step.token_start, step.lengths, table, max_new=most,
                              max_length=min(longest, prompt + i))
        lengths, state = step.lengths, step.free_state
        problems |= step.status | bad
        if i + 1 < steps:
            added = torch.where(lengths > 0, 1, 0).to(torch.int32)
            if i % 5 == 4:
                added[i // 5 % requests] = -1
            tokens, most = requests, 1
    worst = check(cache, q, step.token_start, lengths, table, out)
    print(f"{steps} steps of {requests} requests, {int((lengths > 0).sum())} left, longest {int(lengths.max())} tokens, "
          f"{int(state[1])} of {blocks} blocks free; status {int(problems)}; "
          f"last step within {worst:.2g} of attention over the loaded cache")
    return int(problems), worst


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=16)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--code", choices=("q8", "e4m3"), default="q8")
    a = p.parse_args()
    main(a.requests, a.steps, a.code)
