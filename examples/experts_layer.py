#!/usr/bin/env python3
"""A layer of experts in E4M3 blocks: a router's choices, gate and up projections, down projection, back to the tokens.

The weights are rounded to tiles of 128 x 128 once, as when a model is loaded.  Every step is four calls on the GPU with
no copy to the host: moe_sort puts the (token, choice) pairs in the experts' order, moe_gemm_fp8_block multiplies each
expert's rows with its weight (first the tokens' rows, with silu(gate) * up as its epilogue, then the sorted rows),
moe_combine weights and sums them.  The layer's last step is compared with the same products of the codes' values, and the
gradient of the router's shares with the formula.

Usage: python examples/experts_layer.py [--tokens 64] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_nq_amd as nq  # noqa: E402

HIDDEN, INNER, EXPERTS, TOP = 1024, 512, 16, 4


def check(x, ids, share, w13, w2, h, rows, plan, out):
    """Largest difference from the products of the codes' values, relative to the largest output."""
    values = lambda codes, scales, tile: nq.dequantize_fp8_block(codes, scales, tile)  # noqa: E731
    a, b = (values(w.codes, w.scales, nq.FP8_BLOCK) for w in (w13, w2))
    xv, hv = (values(*nq.quantize_fp8_block(v), 1) for v in (x, h))
    worst = 0.0
    for t in range(min(8, x.shape[0])):
        want = torch.zeros(HIDDEN, device=x.device)
        for c in range(TOP):
            e, p = int(ids[t, c]), int(plan.places[t, c])
            gate, up = (a[e] @ xv[t]).split(INNER)
            worst = max(worst, float((h[p].float() - torch.nn.functional.silu(gate) * up).abs().max() / h.float().abs().max()))
            want += share[t, c] * (b[e] @ hv[p])
        worst = max(worst, float((out[t].float() - want).abs().max() / out.float().abs().max()))
    grad = torch.randn_like(out)
    _, grad_share = nq.moe_combine_grad(grad, rows, plan, share)
    formula = (grad.float()[:, None] * rows.float()[plan.places.long()]).sum(2)
    return worst, float((grad_share - formula).abs().max() / formula.abs().max())


def main(tokens=64, steps=20, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    w13 = nq.Fp8Weight.quantize(new(EXPERTS, 2 * INNER, HIDDEN) / 32)
    w2 = nq.Fp8Weight.quantize(new(EXPERTS, HIDDEN, INNER) / 24)
    for _ in range(steps):
        x = new(tokens, HIDDEN)
        score = torch.softmax(new(tokens, EXPERTS).float(), 1)
        share, ids = score.topk(TOP, 1)
        plan = nq.moe_sort(ids, EXPERTS)
        h = nq.moe_gemm_fp8_block(w13, x, plan, gated=True)
        rows = nq.moe_gemm_fp8_block(w2, h, plan, sorted_rows=True)
        out = nq.moe_combine(rows, plan, share.contiguous())
    worst, gradient = check(x, ids, share.contiguous(), w13, w2, h, rows, plan, out)
    busy = int((plan.offsets[1:] > plan.offsets[:-1]).sum())
    print(f"{steps} steps of {tokens} tokens, {busy} of {EXPERTS} experts busy in the last; within {worst:.2g} of the products "
          f"of the codes' values, the shares' gradient within {gradient:.2g} of the formula")
    return worst, gradient


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    main(a.tokens, a.steps)
