"""GPU: every instance of the E4M3 products' kernels (tests/fp8_cases.py, whose sizes test_fp8_host.py checks against the plan).

Every output is compared with a binary32 matrix product of the codes' values, within the sums' bounds on both sides; some rows
and columns with the definition in binary64, within the kernels' bound alone (fp8_ref); and scales whose product leaves
binary32, on a block of zeros, must not change a bit: that takes the tiles a second way."""
import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import fp8_ref
from fp8_cases import EXPERTS, FAR, FAR_EXPERTS, FEW, FEW_EXPERTS, PRODUCTS
from gpu_util import announce
from test_gpu_fp8_block import DEV, DT, handle, up, values, weight
from test_gpu_moe import choices

pytestmark = pytest.mark.gpu


def large_weight(rng, *shape):
    """Code words of a run of a million and three, which lines up with no row; scales."""
    words, _ = weight(rng, 1, 1000064)
    scales = np.exp(rng.normal(0, 0.5, (*shape[:-2], -(-shape[-2] // 128), shape[-1] // 128))).astype(np.float32) * np.float32(5e-4)
    return np.resize(words[0, :1000003], shape), scales


def numbers(codes, scales, tile):
    return nq.dequantize_fp8_block(codes, scales, tile)


def reference(x, w, gated, wide_sums):
    """The product of two binary32 matrices of values and the bound on the difference of a kernel's output before it is
    rounded: the library's sum of K products (K * 2^-24 of the sum of magnitudes), both sides' values (one rounding each),
    and the kernel's (fp8_ref.product; 7 * 2^-13 covers what the 8-bit instruction drops, whose largest products are a part
    of the magnitudes)."""
    k = x.shape[1]
    y, env = (x @ w.T).double(), (x.abs() @ w.abs().T).double()
    bound = env * ((k + 4) * 2.0 ** -24 + 128 * 2.0 ** -23 + (k // 128 + 18) * 2.0 ** -24 + (0 if wide_sums else 7 * 2.0 ** -13))
    if not gated:
        return y, bound
    h = y.shape[1] // 2
    g, u, bg, bu = y[:, :h], y[:, h:], bound[:, :h], bound[:, h:]
    s = g / (1 + torch.exp(-g))
    return s * u, 1.1 * bg * (u.abs() + bu) + s.abs() * bu + 8 * 2.0 ** -24 * (s * u).abs() + g.abs() * 2.0 ** -23 * (s * u).abs()


def close(y, want, bound, what):
    off = (y.double() - want).abs()
    most = bound + fp8_ref.HALF[y.dtype] * (want.abs() + bound) + fp8_ref.LEAST[y.dtype]
    bad = ~(off <= most)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}"


def sampled(rng, most, count):
    return np.unique(np.r_[0, most - 1, rng.integers(0, most, count)])


def exact(rng, y, xw, xs, ww, ws, gated, wide_sums, what, rows=None):
    """Some rows and columns in binary64; `rows`: those of y, which are xw's in this order."""
    rows = sampled(rng, y.shape[0], 10) if rows is None else rows
    cols = sampled(rng, y.shape[1], 14)
    pick = np.concatenate([cols, cols + y.shape[1]]) if gated else cols
    parts = [fp8_ref.product(xw, xs, ww[c:c + 1], ws[c // 128:c // 128 + 1], wide_sums) for c in pick]
    want = tuple(np.concatenate([p[i] for p in parts], 1) for i in range(2))
    got = y[torch.as_tensor(rows, device=DEV)][:, torch.as_tensor(cols, device=DEV)]
    fp8_ref.check(got, *(fp8_ref.gate(*want) if gated else want), what)


def words_of(codes, rows):
    return codes.view(torch.uint8)[torch.as_tensor(rows, device=DEV)].cpu().numpy()


def far_rows(codes):
    """The same rows 16 MiB apart."""
    base = torch.empty((codes.shape[0], 1 << 24), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    wide = base[:, 64:64 + codes.shape[1]]
    wide.copy_(codes)
    return wide


def product_run(m, n, kb, gated, wide, far=False):
    rng = np.random.default_rng(m + n + kb)
    k = 128 * kb
    ww, ws = large_weight(rng, n, k)
    w = handle(ww, ws)
    w32 = numbers(w.codes, w.scales, 128)
    for dtype in ("f32",) if wide else ("bf16", "f16"):
        announce(f"instance {m} x [{n}, {k}] gated {gated} -> {dtype}{' far' if far else ''}")
        x = values(rng, m, k, dtype, 0.3).to(DEV)
        codes, scales = nq.quantize_fp8_block(x)
        there = far_rows(codes) if far else codes
        # values rounded within the call, but codes where they have to be given
        y = nq.gemm_fp8_block(w, there, scales, bool(gated), DT[dtype]) if far or dtype == "f16" else nq.gemm_fp8_block(w, x, gated=bool(gated))
        close(y, *reference(numbers(codes, scales, 1), w32, gated, wide), f"{m} x [{n}, {k}] {dtype}")
        rows = sampled(rng, m, 10)
        exact(rng, y, words_of(codes, rows), scales[torch.as_tensor(rows, device=DEV)].cpu().numpy(), ww, ws, gated, wide, "exact", rows)
        beyond(rng, w, there, scales, gated, DT[dtype])


def beyond(rng, w, codes, scales, gated, out, plan=None, is_sorted=False):
    """The last block's codes of x become zeros (in place): its scales do not matter then."""
    run = (lambda v, s: nq.gemm_fp8_block(v, codes, s, bool(gated), out)) if plan is None else \
        (lambda v, s: nq.moe_gemm_fp8_block(v, codes, plan, s, is_sorted, bool(gated), out))
    codes.view(torch.uint8)[:, -128:] = 0
    want = run(w, scales)
    assert bool(want.isfinite().all())
    xs, ws = scales.clone(), w.scales.clone()
    xs[:, -1], ws[..., -1] = 2.0 ** 100, 2.0 ** 90
    assert torch.equal(run(nq.Fp8Weight(w.codes, ws), xs), want), "scales of a block of zeros changed the result"


@pytest.mark.parametrize("m, n, kb, gated, wide", PRODUCTS)
def test_products(m, n, kb, gated, wide):
    product_run(m, n, kb, gated, wide)


@pytest.mark.parametrize("m, n, kb, gated, wide", FAR)
def test_products_of_far_rows(m, n, kb, gated, wide):
    product_run(m, n, kb, gated, wide, True)


@pytest.mark.parametrize("m, n, kb, gated", FEW)
def test_few_rows(m, n, kb, gated):
    rng = np.random.default_rng(m + n + kb)
    k = 128 * kb
    ww, ws = large_weight(rng, n, k)
    w = handle(ww, ws)
    w32 = numbers(w.codes, w.scales, 128)
    for dtype in DT:
        announce(f"few rows {m} x [{n}, {k}] gated {gated} {dtype}")
        x = values(rng, m, k, dtype, 0.3).to(DEV)
        codes, scales = nq.quantize_fp8_block(x)
        want = reference(numbers(codes, scales, 1), w32, gated, True)
        for y in (nq.gemm_fp8_block(w, x, gated=bool(gated)), nq.gemm_fp8_block(w, codes, scales, bool(gated), DT[dtype])):
            close(y, *want, f"{m} x [{n}, {k}] {dtype}")
            rows = np.arange(m)
            exact(rng, y, words_of(codes, rows), scales.cpu().numpy(), ww, ws, gated, True, "exact", rows)
        zeros = x.clone()
        zeros[:, -128:] = 0
        beyond(rng, w, codes, scales, gated, DT[dtype])
        # values: the last block's scale is 2^-126, the weight's as large as it can be; the one before it leaves binary32
        big, ws2 = zeros.float() if dtype == "f16" else zeros, w.scales.clone()
        if kb > 1:
            big[:, -256:-128] = 0
            big[:, -256] = 2.0 ** 120
            ws2[..., -2] = 2.0 ** 20
            w2 = w.codes.clone()
            w2.view(torch.uint8)[..., -256] = 0
            w0 = nq.Fp8Weight(w2, ws2)
            got = nq.gemm_fp8_block(w0, big, gated=bool(gated), out_dtype=DT[dtype])
            big[:, -256] = 0
            assert torch.equal(got, nq.gemm_fp8_block(w0, big, gated=bool(gated), out_dtype=DT[dtype]))


def experts_run(tokens, top, experts, n, kb, gated, wide, few, far=False):
    rng = np.random.default_rng(tokens + n + kb)
    k = 128 * kb
    ww, ws = large_weight(rng, experts, n, k)
    w = handle(ww, ws)
    for kind, is_sorted, dtype in (("random", False, "bf16"), ("half", True, "f16"), ("one", False, "bf16")):
        out = "f32" if wide else dtype
        if few and kind == "half" and gated:
            out = "bf16"
        announce(f"instance {tokens} x {top} of {experts} [{n}, {k}] gated {gated} {kind} -> {out}{' far' if far else ''}")
        plan = nq.moe_sort(torch.as_tensor(choices(rng, tokens, top, experts, kind), device=DEV), experts)
        x = values(rng, tokens * top if is_sorted else tokens, k, dtype, 0.3).to(DEV)
        codes, scales = nq.quantize_fp8_block(x)
        there = far_rows(codes) if far else codes
        if far or is_sorted:
            y = nq.moe_gemm_fp8_block(w, there, plan, scales, is_sorted, bool(gated), DT[out])
        else:
            y = nq.moe_gemm_fp8_block(w, x, plan, gated=bool(gated), out_dtype=DT[out])
        x32 = numbers(codes, scales, 1)
        order, offsets = plan.order.cpu().numpy(), plan.offsets.cpu().numpy()
        for e in range(experts):
            at = np.arange(offsets[e], offsets[e + 1])
            if at.size == 0:
                continue
            rows = at if is_sorted else order[at] // top
            w32 = numbers(w.codes[e], w.scales[e], 128)
            part = y[int(offsets[e]):int(offsets[e + 1])]
            close(part, *reference(x32[torch.as_tensor(rows, device=DEV)], w32, gated, wide or few), f"expert {e} {kind}")
            if e in (0, experts // 2, experts - 1):
                some = sampled(rng, at.size, 4)
                exact(rng, part, words_of(codes, rows[some]), scales[torch.as_tensor(rows[some], device=DEV)].cpu().numpy(), ww[e], ws[e], gated,
                      wide or few, f"expert {e} {kind}", some)
        assert not bool(y[int(offsets[-1]):].any())
        beyond(rng, w, there, scales, gated, DT[out], plan, is_sorted)


@pytest.mark.parametrize("tokens, top, experts, n, kb, gated, wide", EXPERTS)
def test_experts(tokens, top, experts, n, kb, gated, wide):
    experts_run(tokens, top, experts, n, kb, gated, wide, False)


@pytest.mark.parametrize("tokens, top, experts, n, kb, gated, wide", FAR_EXPERTS)
def test_experts_of_far_rows(tokens, top, experts, n, kb, gated, wide):
    experts_run(tokens, top, experts, n, kb, gated, wide, False, True)


@pytest.mark.parametrize("tokens, top, experts, n, kb, gated", FEW_EXPERTS)
def test_experts_of_few_rows(tokens, top, experts, n, kb, gated):
    experts_run(tokens, top, experts, n, kb, gated, False, True)
