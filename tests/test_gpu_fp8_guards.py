"""GPU: the E4M3 block and experts' calls of the C ABI write nothing outside of their outputs and workspaces and use nothing
outside of their inputs, for plans that a sort gives and for plans of any words."""
import ctypes

import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import fp8_ref
from gpu_util import announce
from guarded import Guarded, given
from test_gpu_fp8_block import DT, values, weight
from test_gpu_moe import choices

pytestmark = pytest.mark.gpu
CODE = {"f32": 0, "f16": 1, "bf16": 2}


def stream():
    return torch.cuda.current_stream().cuda_stream


def words(rng, tokens, *shape):
    """Places and offsets that no sort gives."""
    return rng.choice([-2 ** 31, -7, -1, 0, 3, tokens - 1, tokens, 2 * tokens - 1, 2 * tokens, 2 ** 31 - 1], shape).astype(np.int32)


class Plan:
    def __init__(self, order, places, offsets):
        self.parts = [given(v, torch.int32) for v in (order, places, offsets)]
        self.tokens, self.top = places.shape
        self.experts = offsets.size - 1
        self.desc = nq.MoePlanDesc(*[p.ptr for p in self.parts], self.tokens, self.top, self.experts)
        self.ref = ctypes.byref(self.desc)

    def check(self, what):
        for p in self.parts:
            p.check(what)


def plans(rng, tokens, top, experts):
    """Plans of a sort and of any words, with what they are."""
    for kind in ("random", "half", "few"):
        yield kind, Plan(*fp8_ref.sort(choices(rng, tokens, top, experts, kind), experts))
    for i in range(3):
        yield f"any words {i}", Plan(words(rng, tokens, tokens * top), words(rng, tokens, tokens, top), words(rng, tokens, experts + 1))


def product(x, xs, w, ws, n, k, gated, out, plan=None, is_sorted=False):
    """nq_gemm_fp8_block with a workspace of just the bytes that it asks for; the output, checked and finite."""
    rows = x.tensor.shape[0]
    out_rows = rows if plan is None else plan.tokens * plan.top
    y = Guarded((out_rows, n // 2 if gated else n), DT[out])
    x_type = 0 if xs is not None else {v: CODE[t] for t, v in DT.items()}[x.tensor.dtype]
    args = nq.Fp8BlockArgs(x.ptr, k, xs.ptr if xs else None, w.ptr, ws.ptr, y.ptr, rows, n, k, x_type, CODE[out], gated, is_sorted)
    need, lib, ref = ctypes.c_uint64(), nq.library(), plan.ref if plan else None
    assert lib.nq_gemm_fp8_block_workspace(ctypes.byref(args), ref, need) == 0
    room = Guarded((need.value,), torch.uint8)
    st = lib.nq_gemm_fp8_block(ctypes.byref(args), ref, room.ptr if need.value else None, need.value, stream())
    assert st == 0
    torch.cuda.synchronize()
    for g, what in ((y, "output"), (room, "workspace"), (x, "x"), (xs, "scales of x"), (w, "weight"), (ws, "scales of the weight"), (plan, "plan")):
        if g is not None:
            g.check(what)
    assert bool(y.tensor.isfinite().all())
    return y.tensor


@pytest.mark.parametrize("m, n, k, gated", [(1, 1, 128, False), (3, 130, 384, False), (16, 24832, 128, True), (17, 257, 1152, False), (40, 256, 8192, True),
                                            (77, 515, 1152, False), (300, 1027, 256, False), (522, 13312, 128, True), (399, 8900, 256, False)])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_products_stay_inside(m, n, k, gated, out):
    rng = np.random.default_rng(m)
    ww, ws = weight(rng, n, k)
    if out == "f16":
        ws *= np.float32(1e-3)  # (the sums of the largest calls stay in binary16's range)
    w, s = given(ww, torch.float8_e4m3fn), given(ws, torch.float32)
    for dtype in ("f32", "bf16"):
        announce(f"guarded product {m} x [{n}, {k}] {dtype} -> {out}")
        x = values(rng, m, k, dtype, 0.3) * 0.05
        a = product(given(x, DT[dtype]), None, w, s, n, k, gated, out)
        xw, xs = fp8_ref.quantize(x.float().numpy())
        b = product(given(xw, torch.float8_e4m3fn), given(xs, torch.float32), w, s, n, k, gated, out)
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens, top, experts, n, k", [(1, 1, 1, 256, 128), (6, 2, 5, 256, 128), (90, 2, 5, 512, 2304), (400, 2, 5, 256, 128),
                                                         (300, 6, 70, 256, 1408), (700, 8, 12, 1536, 256)])
def test_experts_products_stay_inside(tokens, top, experts, n, k):
    rng = np.random.default_rng(tokens)
    ww, ws = weight(rng, experts, n, k)
    w, s = given(ww, torch.float8_e4m3fn), given(ws, torch.float32)
    for what, plan in plans(rng, tokens, top, experts):
        for gated, is_sorted, out in ((False, False, "bf16"), (True, True, "f32"), (True, False, "bf16")):
            announce(f"guarded experts {tokens} x {top} of {experts} [{n}, {k}] {what} gated {gated} sorted {is_sorted}")
            x = values(rng, tokens * top if is_sorted else tokens, k, "bf16", 0.3) * 0.05
            product(given(x, torch.bfloat16), None, w, s, n, k, gated, out, plan, is_sorted)


@pytest.mark.parametrize("tokens, top, cols", [(1, 1, 1), (37, 5, 7), (37, 5, 64), (4100, 3, 136), (4111, 3, 30), (1031, 3, 1024), (6, 2, 5000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_stay_inside(tokens, top, cols, dtype):
    rng = np.random.default_rng(cols)
    t, lib = DT[dtype], nq.library()
    size = torch.empty((), dtype=t).element_size()
    x, rows = (given(torch.as_tensor(rng.normal(0, 1, (r, cols)), dtype=t), t) for r in (tokens, tokens * top))
    share = given(rng.random((tokens, top)).astype(np.float32), torch.float32)
    for what, plan in plans(rng, tokens, top, 12):
        announce(f"guarded rows {tokens} x {top} of {cols} {dtype} {what}")
        gathered, summed, grads = (Guarded((r, cols), t) for r in (tokens * top, tokens, tokens * top))
        grad_share = Guarded((tokens, top), torch.float32)
        assert lib.nq_moe_gather(plan.ref, x.ptr, cols * size, cols * size, gathered.ptr, stream()) == 0
        assert lib.nq_moe_combine(plan.ref, rows.ptr, cols, CODE[dtype], cols, share.ptr, summed.ptr, stream()) == 0
        assert lib.nq_moe_combine_grad(plan.ref, x.ptr, cols, rows.ptr, cols, CODE[dtype], cols, share.ptr, grads.ptr, grad_share.ptr, stream()) == 0
        torch.cuda.synchronize()
        for g, name in ((gathered, "gather"), (summed, "combine"), (grads, "gradient of rows"), (grad_share, "gradient of weights"), (x, "x"),
                        (rows, "rows"), (share, "weights"), (plan, "plan")):
            g.check(f"{what}, {name}")
        for g in (gathered, summed, grads, grad_share):
            assert bool(g.tensor.isfinite().all()), what


@pytest.mark.parametrize("tokens, top, experts", [(1, 1, 1), (5, 8, 64), (171, 3, 200), (4097, 1, 1024), (5000, 8, 60)])
def test_sorts_stay_inside(tokens, top, experts):
    rng, lib = np.random.default_rng(tokens), nq.library()
    for wide in (0, 1):
        ids = choices(rng, tokens, top, experts, "half")
        data = torch.as_tensor(ids, dtype=torch.int64 if wide else torch.int32)
        src = Guarded(data.shape, data.dtype, data, 0)  # (pairs of expert 0 on both sides)
        order, places, offsets = (Guarded(s, torch.int32) for s in ((tokens * top,), (tokens, top), (experts + 1,)))
        need = ctypes.c_uint64()
        assert lib.nq_moe_sort_workspace(tokens, top, experts, need) == 0
        room = Guarded((need.value,), torch.uint8)
        assert lib.nq_moe_sort(src.ptr, wide, tokens, top, experts, order.ptr, places.ptr, offsets.ptr, room.ptr if need.value else None,
                               need.value, stream()) == 0
        torch.cuda.synchronize()
        for g, name, want in zip((order, places, offsets), ("order", "places", "offsets"), fp8_ref.sort(ids, experts)):
            g.check(name)
            assert np.array_equal(g.tensor.cpu().numpy(), want), name
        src.check("ids")
        room.check("workspace")


@pytest.mark.parametrize("rows, cols", [(1, 128), (7, 384), (129, 256), (300, 1152)])
@pytest.mark.parametrize("tile", [1, 128])
def test_codes_and_values_stay_inside(rows, cols, tile):
    rng, lib = np.random.default_rng(rows), nq.library()
    for dtype in DT:
        x = values(rng, 2 * rows, cols, dtype).view(2, rows, cols)
        src = given(x, DT[dtype])
        codes = Guarded((2, rows, cols), torch.uint8)
        scales = Guarded((2, -(-rows // tile), cols // 128), torch.float32)
        assert lib.nq_quantize_fp8_block(src.ptr, CODE[dtype], 2, rows, cols, cols, tile, codes.ptr, scales.ptr, stream()) == 0
        torch.cuda.synchronize()
        for g, name in ((src, "x"), (codes, "codes"), (scales, "scales")):
            g.check(name)
        for i in range(2):
            w, s = fp8_ref.quantize(x[i].float().numpy(), tile)
            assert np.array_equal(codes.tensor[i].cpu().numpy(), w) and np.array_equal(scales.tensor[i].cpu().numpy(), s)
        a, b = given(codes.tensor, torch.uint8), given(scales.tensor, torch.float32)
        back = Guarded((2, rows, cols), DT[dtype])
        assert lib.nq_dequantize_fp8_block(a.ptr, b.ptr, 2, rows, cols, tile, CODE[dtype], back.ptr, stream()) == 0
        torch.cuda.synchronize()
        for g, name in ((a, "codes"), (b, "scales"), (back, "values")):
            g.check(name)
        assert bool(back.tensor.isfinite().all())
