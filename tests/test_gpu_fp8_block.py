"""GPU: E4M3 blocks of 128 (quantize, values, products) against plain implementations (tests/fp8_ref.py).

Quantizing and values are compared exactly: their definition fixes every rounding.  Products are held to the error bound
of their arithmetic (fp8_ref.product).
"""
import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import fp8_ref
from gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def values(rng, rows, cols, dtype, spread=1.0):
    """Rows of different size, some columns larger, some zeros."""
    x = rng.normal(0, 1, (rows, cols)) * np.exp(rng.normal(0, spread, (rows, 1)))
    x[:, ::61] *= 20
    x[rng.random((rows, cols)) < 0.02] = 0
    return torch.as_tensor(x, dtype=torch.float32).to(DT[dtype])


def weight(rng, *shape):
    """Code words (no NaN) and scales."""
    w = rng.integers(0, 256, shape, dtype=np.uint8)
    w[(w & 127) == 127] ^= 1
    w[(w & 0x78) == 0x78] &= 0xBF  # most codes below 2^4, some at the ends of the range
    w[..., 5::37] |= 0x40
    w[(w & 127) == 127] ^= 1
    s = np.exp(rng.normal(0, 0.5, (*shape[:-2], -(-shape[-2] // 128), shape[-1] // 128))).astype(np.float32) * np.float32(0.01)
    return w, s


def up(words):
    return torch.as_tensor(words, device=DEV).view(torch.float8_e4m3fn)


def handle(w, s):
    return nq.Fp8Weight(up(w), torch.as_tensor(s, device=DEV))


def same_codes(codes, words, what):
    """Equal words, any NaN word for a NaN."""
    got = codes.detach().cpu().view(torch.uint8).numpy()
    nan = (words & 127) == 127
    assert np.array_equal((got & 127) == 127, nan), f"{what}: NaN codes"
    assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, words)), f"{what}: codes"


# --- codes ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("rows, cols", [(1, 128), (7, 384), (127, 128), (128, 256), (129, 128), (300, 1152), (3, 16384)])
def test_quantize_and_values(rows, cols, tile, dtype):
    rng = np.random.default_rng(rows + cols + tile)
    x = values(rng, rows, cols, dtype)
    announce(f"quantize_fp8_block [{rows}, {cols}] tile {tile} {dtype}")
    codes, scales = nq.quantize_fp8_block(x.to(DEV), tile)
    words, want = fp8_ref.quantize(x.float().numpy(), tile)
    assert np.array_equal(scales.cpu().numpy(), want)
    same_codes(codes, words, "quantize")
    exact = fp8_ref.numbers(words, want, tile)
    for out in DT.values():
        y = nq.dequantize_fp8_block(codes, scales, tile, out)
        rounded = torch.as_tensor(exact).to(torch.float32).to(out)  # a product of 28 bits rounds to binary32 first
        assert torch.equal(y.cpu(), rounded)


def test_quantize_ends_of_the_range():
    x = np.zeros((8, 256), np.float32)
    x[0, :128] = np.float32(3.4028235e38)          # the largest
    x[1, 3] = np.float32(1e-45)                    # the least subnormal
    x[2, :] = np.linspace(-1e-38, 1e-38, 256)      # scales below 2^-126
    x[3, 5], x[3, 200] = np.inf, -np.inf           # not finite among finite ones
    x[3, 6] = 2.0
    x[4, 7] = np.nan
    x[4, 8] = -3.0
    x[5, :128] = np.nan                            # nothing finite
    x[6, :] = 448 * np.where(np.arange(256) % 2, 1, -1)
    x[7, :] = np.arange(256) - 128                 # ties
    for tile in (1, 128):
        codes, scales = nq.quantize_fp8_block(torch.as_tensor(x, device=DEV), tile)
        words, want = fp8_ref.quantize(x, tile)
        assert np.array_equal(scales.cpu().numpy(), want)
        same_codes(codes, words, f"ends, tile {tile}")
        y = nq.dequantize_fp8_block(codes, scales, tile).cpu().numpy()
        assert np.array_equal(np.isnan(y), ~np.isfinite(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_strides_and_addresses(dtype):
    rng = np.random.default_rng(3)
    base = values(rng, 40, 700, dtype)
    wide = base.to(DEV)
    for x, what in ((wide[:, 8:8 + 256], "slice"), (wide[:, 3:3 + 256], "odd address"), (wide[5:6, 16:144].expand(9, 128), "one row for all")):
        ref = x.cpu().float().numpy()
        for tile in (1, 128):
            codes, scales = nq.quantize_fp8_block(x, tile)
            words, want = fp8_ref.quantize(np.ascontiguousarray(ref), tile)
            assert np.array_equal(scales.cpu().numpy(), want), what
            same_codes(codes, words, what)


@pytest.mark.parametrize("rows", [1, 100, 128, 130, 257])
def test_quantize_several_matrices(rows):
    rng = np.random.default_rng(rows)
    x = values(rng, 3 * rows, 256, "bf16").view(3, rows, 256)
    for tile in (1, 128):
        codes, scales = nq.quantize_fp8_block(x.to(DEV), tile)
        y = nq.dequantize_fp8_block(codes, scales, tile).cpu().numpy()
        for i in range(3):
            words, want = fp8_ref.quantize(x[i].float().numpy(), tile)
            assert np.array_equal(scales[i].cpu().numpy(), want)
            same_codes(codes[i], words, f"matrix {i}")
            assert np.array_equal(y[i], fp8_ref.numbers(words, want, tile).astype(np.float32))


# --- products ---------------------------------------------------------------------------------------------------

def run(rng, m, n, k, dtype, out, gated, codes, what=""):
    x = values(rng, m, k, dtype, 0.5)
    ww, ws = weight(rng, n, k)
    announce(f"gemm_fp8_block {m} x [{n}, {k}] {dtype} -> {out} gated {gated} codes {codes} {what}")
    w, xd = handle(ww, ws), x.to(DEV)
    if codes:
        y = nq.gemm_fp8_block(w, *nq.quantize_fp8_block(xd), gated=gated, out_dtype=DT[out])
    else:
        y = nq.gemm_fp8_block(w, xd, gated=gated, out_dtype=DT[out])
    torch.cuda.synchronize()
    want = fp8_ref.product(*fp8_ref.quantize(x.float().numpy()), ww, ws, out == "f32" or fp8_ref.few_rows(m))
    fp8_ref.check(y, *(fp8_ref.gate(*want) if gated else want), f"{m} x [{n}, {k}]")
    return x, w, y


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n, k, gated", [(1, 128, False), (30, 384, False), (129, 1152, False), (256, 128, True), (512, 640, True)])
def test_few_rows(m, n, k, gated):
    rng = np.random.default_rng(m * n)
    run(rng, m, n, k, ("f32", "f16", "bf16")[m % 3], ("bf16", "f32")[n % 2], gated, m % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [3, 40, 70])
def test_types(m, dtype, out):
    rng = np.random.default_rng(m)
    for codes in (False, True):
        run(rng, m, 144, 256, dtype, out, False, codes)


@pytest.mark.parametrize("m, n, k", [(65, 1, 128), (65, 130, 2048), (77, 515, 1152), (128, 128, 4096), (129, 256, 384), (257, 130, 640), (300, 384, 128), (300, 1027, 256)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_many_rows(m, n, k, out):
    rng = np.random.default_rng(m + n)
    run(rng, m, n, k, "bf16", out, False, m % 2 == 0)


@pytest.mark.parametrize("m, n, k", [(65, 256, 1024), (130, 768, 384), (300, 512, 256)])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_many_rows_gated(m, n, k, out):
    rng = np.random.default_rng(m + n)
    run(rng, m, n, k, "f16", out, True, m % 2 == 0)


@pytest.mark.parametrize("m, n, gated, out", [(4200, 4100, False, "bf16"), (4200, 4099, False, "f16"), (4111, 8192, True, "bf16"), (4111, 4096, False, "f32")])
def test_largest_tiles(m, n, gated, out):
    """Sizes that fill the device with the largest tiles; some rows and columns of them are compared."""
    rng = np.random.default_rng(m)
    k = 256
    x = values(rng, m, k, "bf16", 0.5)
    ww, ws = weight(rng, n, k)
    announce(f"gemm_fp8_block {m} x [{n}, {k}] gated {gated}")
    y = nq.gemm_fp8_block(handle(ww, ws), x.to(DEV), gated=gated, out_dtype=DT[out])
    torch.cuda.synchronize()
    no = n // 2 if gated else n
    rows = np.unique(np.r_[0, 255, 256, m - 1, rng.integers(0, m, 40)])
    cols = np.unique(np.r_[0, 127, 128, no - 1, rng.integers(0, no, 60)])
    xw, xs = fp8_ref.quantize(x.float().numpy()[rows])
    pick = np.concatenate([cols, cols + no]) if gated else cols
    # each picked weight row with the scales of its own tile
    ww_p, ws_p = ww[pick], ws[pick // 128]
    parts = [fp8_ref.product(xw, xs, ww_p[i:i + 1], ws_p[i:i + 1], out == "f32") for i in range(pick.size)]
    want = tuple(np.concatenate([p[j] for p in parts], 1) for j in range(2))
    got = y[torch.as_tensor(rows, device=DEV)][:, torch.as_tensor(cols, device=DEV)]
    fp8_ref.check(got, *(fp8_ref.gate(*want) if gated else want), "largest tiles")
    assert bool(y.isfinite().all())


@pytest.mark.parametrize("m", [1, 9, 16, 40, 100])
def test_values_and_codes_give_the_same_bits(m):
    rng = np.random.default_rng(m)
    x, w, y = run(rng, m, 144, 1152, "bf16", "f32", False, False)
    again = nq.gemm_fp8_block(w, *nq.quantize_fp8_block(x.to(DEV)), out_dtype=torch.float32)
    assert torch.equal(y, again)
    assert torch.equal(y, nq.gemm_fp8_block(w, x.to(DEV), out_dtype=torch.float32))


@pytest.mark.parametrize("m", [5, 80])
def test_product_strides_and_addresses(m):
    rng = np.random.default_rng(m)
    ww, ws = weight(rng, 50, 256)
    w = handle(ww, ws)
    base = values(rng, m, 700, "bf16", 0.5).to(DEV)
    for x, what in ((base[:, 8:264], "slice"), (base[:, 3:259], "odd address"), (base[1:2, :256].expand(m, 256), "one row for all")):
        want = fp8_ref.product(*fp8_ref.quantize(x.cpu().float().numpy()), ww, ws, m <= 16)
        fp8_ref.check(nq.gemm_fp8_block(w, x), *want, what)
    codes, scales = nq.quantize_fp8_block(base[:, :640].contiguous())
    part = codes[:, 256:512]
    some = scales[:, 2:4].contiguous()
    want = fp8_ref.product(part.cpu().view(torch.uint8).numpy(), some.cpu().numpy(), ww, ws, m <= 16)
    fp8_ref.check(nq.gemm_fp8_block(w, part, some, out_dtype=torch.float16), *want, "codes in wide rows")


@pytest.mark.parametrize("m", [3, 30, 90])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_not_finite_stays_in_its_row_and_column(m, out):
    rng = np.random.default_rng(m)
    x = values(rng, m, 384, "f32", 0.5)
    ww, ws = weight(rng, 70, 384)
    x[1, 200], x[2, 5] = float("nan"), float("inf")
    ww[66, 300] = 0x7F
    y = nq.gemm_fp8_block(handle(ww, ws), x.to(DEV), out_dtype=DT[out]).cpu()
    bad = torch.zeros(m, 70, dtype=torch.bool)
    bad[1:3] = True
    bad[:, 66] = True
    assert torch.equal(y.isnan(), bad)
    clean, ok = x.clone(), ww.copy()
    clean[1, 200], clean[2, 5], ok[66, 300] = 0, 0, 0
    want, bound = fp8_ref.product(*fp8_ref.quantize(clean.numpy()), ok, ws, out == "f32" or m <= 16)
    fp8_ref.check(y, np.where(bad, np.nan, want), bound, "not finite")


def test_extreme_scales():
    """Blocks whose scales are far apart: the sums keep the small ones' precision where the large ones are zero."""
    rng = np.random.default_rng(1)
    for m, out in ((4, torch.float32), (100, torch.float32), (100, torch.bfloat16)):
        x = rng.normal(0, 1, (m, 512)).astype(np.float32)
        x[:, 128:256] = 0
        x[:, 256:384] *= np.float32(1e-30)
        x[::2, :128] *= np.float32(1e30)
        ww, ws = weight(rng, 64, 512)
        want = fp8_ref.product(*fp8_ref.quantize(x), ww, ws, m <= 16 or out is torch.float32)
        fp8_ref.check(nq.gemm_fp8_block(handle(ww, ws), torch.as_tensor(x, device=DEV), out_dtype=out), *want, "extreme scales")


def test_codes_beyond_32_bits_of_the_first():
    """Rows of codes 16 MiB apart, the last of them past 2^32 bytes."""
    rng = np.random.default_rng(9)
    m, k, far = 300, 256, 1 << 24
    ww, ws = weight(rng, 130, k)
    w = handle(ww, ws)
    base = torch.empty((m, far), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    codes, scales = nq.quantize_fp8_block(values(rng, m, k, "bf16", 0.5).to(DEV))
    wide = base[:, 32:32 + k]
    wide.copy_(codes)
    for rows in (3, 100, 300):
        for out in (torch.bfloat16, torch.float32):
            announce(f"far codes {rows} {out}")
            want = fp8_ref.product(codes[:rows].cpu().view(torch.uint8).numpy(), scales[:rows].cpu().numpy(), ww, ws,
                                   out is torch.float32 or fp8_ref.few_rows(rows))
            fp8_ref.check(nq.gemm_fp8_block(w, wide[:rows], scales[:rows], out_dtype=out), *want, f"far codes, {rows} rows")


@pytest.mark.parametrize("m", [40, 140])
def test_pieces_of_gated_products(m):
    """K in pieces, few tiles, both halves of the weight in a piece's sums."""
    rng = np.random.default_rng(m)
    run(rng, m, 256, 8192, "bf16", "bf16", True, False)
    run(rng, m, 768, 4096, "bf16", "f32", True, True)


def test_no_rows():
    ww, ws = weight(np.random.default_rng(0), 256, 128)
    w = handle(ww, ws)
    for gated in (False, True):
        y = nq.gemm_fp8_block(w, torch.empty((0, 128), device=DEV), gated=gated)
        assert y.shape == (0, 128 if gated else 256)
    codes, scales = nq.quantize_fp8_block(torch.empty((0, 256), device=DEV))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    assert nq.dequantize_fp8_block(codes, scales).shape == (0, 256)


@pytest.mark.parametrize("m", [4, 50, 200])
def test_other_stream_and_graph(m):
    rng = np.random.default_rng(m)
    x = values(rng, m, 1024, "bf16", 0.5).to(DEV)
    ww, ws = weight(rng, 384, 1024)
    w = handle(ww, ws)
    want = nq.gemm_fp8_block(w, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = nq.gemm_fp8_block(w, x, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    fixed = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nq.gemm_fp8_block(w, fixed)
    for i in range(4):
        new = values(np.random.default_rng(i), m, 1024, "bf16", 0.5).to(DEV)
        eager = nq.gemm_fp8_block(w, new)
        fixed.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), f"replay {i}"


def test_refusals():
    rng = np.random.default_rng(0)
    ww, ws = weight(rng, 192, 256)
    w = handle(ww, ws)
    x = torch.zeros((4, 256), device=DEV)
    with pytest.raises(ValueError):
        nq.gemm_fp8_block(w, x[:, :128])
    with pytest.raises(ValueError):
        nq.gemm_fp8_block(w, x.t().contiguous().t())
    with pytest.raises(ValueError):
        nq.gemm_fp8_block(w, x, torch.zeros((4, 2), device=DEV))
    with pytest.raises(ValueError):
        nq.gemm_fp8_block(w, x.to(torch.float8_e4m3fn), torch.zeros((4, 3), device=DEV))
    with pytest.raises(nq.NqError):
        nq.gemm_fp8_block(w, x, gated=True)  # 192 rows
    with pytest.raises((nq.NqError, KeyError)):
        nq.gemm_fp8_block(w, x, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        nq.Fp8Weight(up(ww), torch.zeros((1, 2), device=DEV))
    with pytest.raises(ValueError):
        nq.Fp8Weight(up(ww)[:, :200], torch.zeros((2, 1), device=DEV))
    with pytest.raises(nq.NqError):
        nq.quantize_fp8_block(x[:, :100])
    with pytest.raises(ValueError):
        nq.quantize_fp8_block(x, tile=64)
    with pytest.raises(ValueError):
        nq.quantize_fp8_block(x.cpu())
