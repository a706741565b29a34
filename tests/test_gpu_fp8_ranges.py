"""GPU: products of E4M3 blocks at the ends of binary32's range, in every kernel: scales whose product leaves it, gates far
below zero."""
import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import fp8_ref
from gpu_util import announce
from test_gpu_fp8_block import DEV, DT, up, weight

pytestmark = pytest.mark.gpu

# rows, N: up to 16 rows, and the many-rows kernel's tiles of 64, 128 (four and two buffers) and 256 (16-bit outputs)
SIZES = [(3, 130), (16, 384), (40, 130), (300, 1027), (370, 5888), (1347, 4100), (2100, 8200)]


def sampled(rng, most, count):
    return np.unique(np.r_[0, most - 1, rng.integers(0, most, count)])


@pytest.mark.parametrize("large_x", [False, True])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m, n", SIZES)
def test_scales_whose_product_leaves_binary32(m, n, out, large_x):
    """The first block's scales are 2^96 and 2^34.  Its codes have one nonzero column: weight rows of 2^-9 where n % 3 is 1
    and of 448 where it is 2, rows of 2^-9 where m % 2 is 0.  So its sums are 0, 2^-18 (2^112 with the scales) or 448 * 2^-9
    (0.875 * 2^130, an infinity)."""
    rng = np.random.default_rng(m + n)
    k = 640
    xw = rng.integers(0, 0x40, (m, k), dtype=np.uint8) | rng.integers(0, 2, (m, k), dtype=np.uint8) << 7
    xs = np.exp(rng.normal(0, 0.5, (m, k // 128))).astype(np.float32)
    ww, ws = weight(rng, n, k)
    xw[:, :128], ww[:, :128] = 0, 0
    xw[::2, 77] = 0x01
    ww[1::3, 77], ww[2::3, 77] = 0x01, 0x7E
    xs[:, 0], ws[:, 0] = (2.0 ** 96, 2.0 ** 34) if large_x else (2.0 ** 34, 2.0 ** 96)
    announce(f"scales beyond binary32 {m} x [{n}, {k}] {out}")
    y = nq.gemm_fp8_block(nq.Fp8Weight(up(ww), torch.as_tensor(ws, device=DEV)), up(xw), torch.as_tensor(xs, device=DEV),
                          out_dtype=DT[out])
    infinite = torch.zeros((m, n), dtype=torch.bool, device=DEV)
    infinite[::2, 2::3] = True
    if out == "f16":  # 2^112 is one there as well
        infinite[::2, 1::3] = True
    assert torch.equal(torch.isposinf(y), infinite) and not bool(y.isnan().any())
    rows, cols = sampled(rng, m, 12), sampled(rng, n, 24)
    parts = [fp8_ref.product(xw[rows], xs[rows], ww[c:c + 1], ws[c // 128:c // 128 + 1], out == "f32" or fp8_ref.few_rows(m))
             for c in cols]
    want, bound = (np.concatenate([p[i] for p in parts], 1) for i in range(2))
    got = y[torch.as_tensor(rows, device=DEV)][:, torch.as_tensor(cols, device=DEV)]
    high = torch.isinf(got).cpu().numpy()
    fp8_ref.check(got.masked_fill(torch.isinf(got), 0), np.where(high, 0, want), np.where(high, 0, bound), "beyond binary32")


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_values_whose_scales_leave_binary32(out):
    """Rows that are values, rounded within the call: weight rows of zeros give zeros, not 0 times an infinity."""
    rng = np.random.default_rng(5)
    for m in (2, 60):
        x = rng.normal(0, 1, (m, 256)).astype(np.float32)
        x[:, :128] *= np.float32(1e37)
        ww, ws = weight(rng, 70, 256)
        ww[::2, :128] = 0
        ws[:, 0] = 1e9
        y = nq.gemm_fp8_block(nq.Fp8Weight(up(ww), torch.as_tensor(ws, device=DEV)), torch.as_tensor(x, device=DEV), out_dtype=DT[out])
        fp8_ref.check(y[:, ::2], *fp8_ref.product(*fp8_ref.quantize(x), ww[::2], ws, out == "f32" or m <= 16), f"{m} rows")


def test_experts_whose_scales_leave_binary32():
    rng = np.random.default_rng(6)
    for tokens, n in ((10, 130), (150, 130), (500, 4100)):
        experts, k = 4, 256
        xw = rng.integers(0, 0x40, (tokens, k), dtype=np.uint8)
        xs = np.ones((tokens, 2), np.float32)
        ww, ws = weight(rng, experts, n, k)
        xw[:, :128] = 0
        xs[:, 0], ws[1:3, :, 0] = 2.0 ** 100, 2.0 ** 60
        plan = nq.moe_sort(torch.as_tensor(rng.integers(0, experts, (tokens, 2)), device=DEV), experts)
        handle = nq.Fp8Weight(up(ww), torch.as_tensor(ws, device=DEV))
        y = nq.moe_gemm_fp8_block(handle, up(xw), plan, torch.as_tensor(xs, device=DEV), out_dtype=torch.bfloat16)
        one = np.where(np.arange(2) == 0, 1, xs).astype(np.float32)  # zeros of a block are zeros whatever its scale
        want = nq.moe_gemm_fp8_block(handle, up(xw), plan, torch.as_tensor(one, device=DEV), out_dtype=torch.bfloat16)
        assert bool(want.isfinite().all()) and torch.equal(y, want)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [1, 16, 17, 200, 2100])
@pytest.mark.parametrize("k", [128, 4096])
def test_gates_far_below_zero(m, k, out):
    """Gates of -60 to -196 and ups of 2^30 to 2^127, each one product of two codes and their scales, so exact: what is
    compared is g / (1 + e^-g) * u alone, e^-g beyond binary32 and e^g below its normal numbers among them.

    The kernels take the fourth root of e^g: a binary32 exponential (1 ulp) in four factors and five roundings for binary32
    outputs and calls of up to 16 rows, 13 * 2^-24; the hardware's exponential, whose argument carries two roundings,
    |g| * 2^-23 more, for others."""
    tiles = 36
    if m == 2100 and k == 4096:
        tiles = 64
    half = 128 * tiles
    g = -np.concatenate([np.linspace(60, 110, 26), np.linspace(115, 196, tiles - 26)]).round()
    u = np.full(tiles, 2.0 ** 127)
    u[:26:2], u[1:26:2] = 2.0 ** 122, 2.0 ** np.arange(30, 121, 7.5).round()  # (silu(-88) is near 2^-120)
    xw, ww = np.zeros((m, k), np.uint8), np.zeros((2 * half, k), np.uint8)
    xw[:, 5], ww[:half, 5], ww[half:, 5] = 0x38, 0xB8, 0x38  # 1, -1 and 1
    ww[:half:5, 5] = 0xB4  # -0.75
    xs, ws = np.ones((m, k // 128), np.float32), np.ones((2 * tiles, k // 128), np.float32)
    ws[:tiles, 0], ws[tiles:, 0] = -g, u
    announce(f"far gates {m} x [{2 * half}, {k}] {out}")
    y = nq.gemm_fp8_block(nq.Fp8Weight(up(ww), torch.as_tensor(ws, device=DEV)), up(xw), torch.as_tensor(xs, device=DEV), gated=True,
                          out_dtype=DT[out])
    gate = np.repeat(g, 128)
    gate[::5] *= 0.75
    with np.errstate(over="ignore"):
        want = gate / (1 + np.exp(-gate)) * np.repeat(u, 128)
    rel = 13 * 2.0 ** -24 + (0 if out == "f32" or fp8_ref.few_rows(m) else np.abs(gate) * 2.0 ** -23)
    want, rel = np.broadcast_to(want, (m, half)), np.broadcast_to(np.abs(want) * rel, (m, half))
    most = {"f32": 3.4e38, "f16": 65504.0, "bf16": 3.38e38}[out]
    inside = np.abs(want) < most
    got = y.masked_fill(torch.as_tensor(~inside, device=DEV), 0)
    fp8_ref.check(got, np.where(inside, want, 0), np.where(inside, rel, 0), "far gates")


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [16, 17, 300])
def test_sums_whose_large_products_cancel(m, out):
    """Of every eight products one is 448 * 448, one -448 * 448 and one 1: the sum is the number of eights.  Up to 16 rows and
    in binary32 outputs it is exact (so each partial sum in binary32 is: multiples of 1 below 2^24).  The 8-bit matrix
    instruction of the others may lose 7 * 2^-13 of the largest product of each eight, here more than the result."""
    n, k = 130, 1152
    xw, ww = np.zeros((m, k), np.uint8), np.zeros((n, k), np.uint8)
    xw[:, 0::8], ww[:, 0::8] = 0x7E, 0x7E
    xw[:, 3::8], ww[:, 3::8] = 0x7E, 0xFE
    xw[:, 6::8], ww[:, 6::8] = 0x38, 0x38
    one = lambda rows: torch.ones((rows, k // 128), device=DEV)  # noqa: E731
    y = nq.gemm_fp8_block(nq.Fp8Weight(up(ww), one(2)), up(xw), one(m), out_dtype=DT[out]).double()
    off = float((y - k // 8).abs().max())
    print(f"{m} rows, {out}: off by {off}")
    if m <= 16 or out == "f32":
        assert off == 0  # 144, which every type holds
    else:
        assert off <= 7 * 2.0 ** -13 * 448 * 448 * (k // 8)
