"""GPU: a router's pairs sorted by expert, the experts' products, and rows back to their tokens with their gradients,
against plain implementations (tests/fp8_ref.py)."""
import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import fp8_ref
from gpu_util import announce
from test_gpu_fp8_block import DT, handle, values, weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def choices(rng, tokens, top, experts, kind="random"):
    if kind == "one":
        return np.full((tokens, top), experts - 1, np.int32)
    if kind == "few":  # most experts have none
        return rng.choice([0, experts // 2, experts - 1], (tokens, top)).astype(np.int32)
    if kind == "half":  # others are elsewhere
        return rng.integers(-experts, 2 * experts, (tokens, top)).astype(np.int32)
    if kind == "none":
        return np.full((tokens, top), -1, np.int32)
    return rng.integers(0, experts, (tokens, top)).astype(np.int32)


def plan_of(ids, experts, wide=False):
    return nq.moe_sort(torch.as_tensor(ids, device=DEV, dtype=torch.int64 if wide else torch.int32), experts)


def same_plan(plan, ids, experts, what):
    for name, a, b in zip(("order", "places", "offsets"), (plan.order, plan.places, plan.offsets), fp8_ref.sort(ids, experts)):
        assert np.array_equal(a.cpu().numpy(), b), f"{what}: {name}"


# --- sort -------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens, top", [(1, 1), (1, 8), (9, 7), (64, 1), (13, 5), (64, 8), (171, 3), (512, 8), (4097, 1), (1366, 3), (5000, 8)])
@pytest.mark.parametrize("experts", [1, 3, 64, 200, 513, 1024])
def test_sort(tokens, top, experts):
    rng = np.random.default_rng(tokens * experts)
    for kind in ("random", "half"):
        ids = choices(rng, tokens, top, experts, kind)
        announce(f"moe_sort {tokens} x {top} of {experts} {kind}")
        same_plan(plan_of(ids, experts, wide=kind == "half"), ids, experts, kind)


@pytest.mark.parametrize("kind", ["one", "few", "none"])
@pytest.mark.parametrize("tokens", [7, 700, 3000])
def test_sort_uneven(kind, tokens):
    ids = choices(np.random.default_rng(tokens), tokens, 4, 60, kind)
    same_plan(plan_of(ids, 60), ids, 60, kind)


def test_sort_of_many_pairs():
    """More than 512 times 4096 pairs: a workgroup takes 8192."""
    ids = np.random.default_rng(8).integers(-1, 41, (700001, 3))
    plan = plan_of(ids, 40, wide=True)
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < 40)
    order = np.argsort(np.where(live, flat, 40), kind="stable")[:live.sum()]
    places = np.full(flat.size, -1)
    places[order] = np.arange(order.size)
    assert np.array_equal(plan.order.cpu().numpy(), np.concatenate([order, np.full(flat.size - order.size, -1)]))
    assert np.array_equal(plan.places.cpu().numpy().reshape(-1), places)
    assert np.array_equal(plan.offsets.cpu().numpy(), np.cumsum([0, *np.bincount(flat[live], minlength=40)]))


def test_copies_of_a_plan():
    """A copy's calls read its own tensors."""
    import copy
    ids = choices(np.random.default_rng(2), 30, 2, 5)
    plan = plan_of(ids, 5)
    other = copy.deepcopy(plan)
    same_plan(other, ids, 5, "copy")
    want = nq.moe_gather(torch.arange(240., device=DEV).view(30, 8), plan)
    for t in (plan.order, plan.places, plan.offsets):
        t.zero_()
    assert torch.equal(nq.moe_gather(torch.arange(240., device=DEV).view(30, 8), other), want)


def test_sort_wide_ids_beyond_32_bits():
    ids = np.array([[2 ** 32, 1], [-2 ** 40, 0], [2 ** 33 + 1, 1]])
    plan = nq.moe_sort(torch.as_tensor(ids, device=DEV), 2)
    same_plan(plan, ids, 2, "wide")


def test_no_tokens():
    plan = nq.moe_sort(torch.empty((0, 4), dtype=torch.int32, device=DEV), 5)
    assert plan.offsets.tolist() == [0] * 6
    assert nq.moe_gather(torch.empty((0, 64), device=DEV), plan).shape == (0, 64)
    rows = torch.empty((0, 64), device=DEV)
    assert nq.moe_combine(rows, plan).shape == (0, 64)
    g, gw = nq.moe_combine_grad(rows, rows, plan, torch.empty((0, 4), device=DEV))
    assert g.shape == (0, 64) and gw.shape == (0, 4)
    ww, ws = weight(np.random.default_rng(0), 5, 32, 128)
    assert nq.moe_gemm_fp8_block(handle(ww, ws), torch.empty((0, 128), device=DEV), plan).shape == (0, 32)


# --- rows -------------------------------------------------------------------------------------------------------

def rows_run(tokens, top, cols, dtype, kind):
    rng = np.random.default_rng(cols)
    experts = 12
    ids = choices(rng, tokens, top, experts, kind)
    plan = plan_of(ids, experts)
    order, places, offsets = fp8_ref.sort(ids, experts)
    t = DT[dtype]
    x = torch.as_tensor(rng.normal(0, 1, (tokens, cols)), dtype=t)
    announce(f"moe rows {dtype} {cols} {kind}")
    got = nq.moe_gather(x.to(DEV), plan).cpu()
    want = torch.where(torch.as_tensor(order >= 0)[:, None], x[torch.as_tensor(np.maximum(order, 0) // top)], torch.zeros((), dtype=t))
    assert torch.equal(got, want)

    rows = torch.as_tensor(rng.normal(0, 1, (tokens * top, cols)), dtype=t)
    rows[offsets[-1]:] = float("nan")  # what lies behind the last place is not read
    w = rng.random((tokens, top)).astype(np.float32)
    r64 = np.where(order[:, None] >= 0, rows.double().numpy(), 0)
    wd = torch.as_tensor(w, device=DEV)
    fp8_ref.check(nq.moe_combine(rows.to(DEV), plan, wd), *fp8_ref.combine(r64, places, w.astype(np.float64)), "combine")
    fp8_ref.check(nq.moe_combine(rows.to(DEV), plan), *fp8_ref.combine(r64, places, np.ones(w.shape)), "combine, no weights")

    grad = torch.as_tensor(rng.normal(0, 1, (tokens, cols)), dtype=t)
    g_rows, g_w = nq.moe_combine_grad(grad.to(DEV), rows.to(DEV), plan, wd)
    want_rows, want_w, bound = fp8_ref.combine_grad(grad.double().numpy(), r64, places, w.astype(np.float64))
    fp8_ref.check(g_rows, want_rows, np.abs(want_rows) * 2.0 ** -24, "gradient of rows")
    fp8_ref.check(g_w, want_w, bound, "gradient of weights")
    g_rows, none = nq.moe_combine_grad(grad.to(DEV), rows.to(DEV), plan)
    assert none is None
    want_rows, _, _ = fp8_ref.combine_grad(grad.double().numpy(), r64, places, np.ones(w.shape))
    fp8_ref.check(g_rows, want_rows, 0 * want_rows, "gradient of rows, no weights")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [1, 7, 8, 64, 2048, 2056, 5000])
@pytest.mark.parametrize("kind", ["random", "half", "none"])
def test_gather_combine_and_gradient(dtype, cols, kind):
    rows_run(37, 5, cols, dtype, kind)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens, cols", [(4100, 8), (4100, 30), (4100, 136), (4111, 256), (1100, 33), (1100, 100), (1031, 264), (1031, 1024)])
def test_narrow_rows_of_many_tokens(tokens, cols, dtype):
    """Several rows a workgroup."""
    rows_run(tokens, 3, cols, dtype, "half")


def test_rows_without_columns():
    rng = np.random.default_rng(0)
    plan = plan_of(choices(rng, 5, 2, 4, "half"), 4)
    rows, w = torch.empty((10, 0), device=DEV), torch.ones((5, 2), device=DEV)
    assert nq.moe_gather(torch.empty((5, 0), device=DEV), plan).shape == (10, 0)
    assert nq.moe_combine(rows, plan, w).shape == (5, 0)
    g, gw = nq.moe_combine_grad(torch.empty((5, 0), device=DEV), rows, plan, w)
    assert g.shape == (10, 0) and not bool(gw.any())


def test_more_bytes_than_the_l2s():
    """Sizes whose rows go past the L2s, and pairs elsewhere."""
    rng = np.random.default_rng(6)
    tokens, top, cols = 3000, 4, 2048
    ids = choices(rng, tokens, top, 20, "half")
    plan = plan_of(ids, 20)
    order, places, offsets = fp8_ref.sort(ids, 20)
    x = torch.as_tensor(rng.normal(0, 1, (tokens, cols)), dtype=torch.bfloat16)
    live = torch.as_tensor(order >= 0)[:, None]
    token = torch.as_tensor(np.maximum(order, 0) // top)
    assert torch.equal(nq.moe_gather(x.to(DEV), plan).cpu(), torch.where(live, x[token], torch.zeros((), dtype=x.dtype)))
    w = torch.as_tensor(rng.random((tokens, top)), dtype=torch.float32)
    rows = torch.zeros((tokens * top, cols), dtype=torch.bfloat16, device=DEV)
    g, _ = nq.moe_combine_grad(x.to(DEV), rows, plan, w.to(DEV))
    per = w.reshape(-1)[torch.as_tensor(np.maximum(order, 0)).long()][:, None]
    want = torch.where(live, (x.float()[token] * per).to(torch.bfloat16), torch.zeros((), dtype=x.dtype))  # one product of two binary32 numbers, rounded twice
    assert torch.equal(g.cpu(), want)


def test_gradients_against_differences():
    """Combining is linear in rows and in weights: a step of any size gives its gradient, up to the sums' rounding."""
    rng = np.random.default_rng(0)
    ids = choices(rng, 20, 3, 8, "half")
    plan = plan_of(ids, 8)
    n = int(plan.offsets[-1])
    rows, w, grad = (torch.as_tensor(rng.normal(0, 1, s), dtype=torch.float32, device=DEV) for s in ((60, 40), (20, 3), (20, 40)))
    g_rows, g_w = nq.moe_combine_grad(grad, rows, plan, w)
    loss = lambda r, v: float((nq.moe_combine(r, plan, v).double() * grad.double()).sum())  # noqa: E731
    # 800 outputs, each off by at most 3 roundings of terms of at most 6 * 4 (normal values), times a gradient of at most 5
    slack = 800 * 3 * 2.0 ** -24 * 24 * 5
    for _ in range(8):
        d, e = (torch.as_tensor(rng.normal(0, 1, s), dtype=torch.float32, device=DEV) for s in ((60, 40), (20, 3)))
        diff = (loss(rows + d, w) - loss(rows - d, w)) / 2
        assert abs(diff - float((g_rows[:n].double() * ((rows + d) - (rows - d))[:n].double() / 2).sum())) <= 8 * slack
        diff = (loss(rows, w + e) - loss(rows, w - e)) / 2
        assert abs(diff - float((g_w.double() * ((w + e) - (w - e)).double() / 2).sum())) <= 8 * slack
    x = torch.as_tensor(rng.normal(0, 1, (20, 40)), dtype=torch.float32, device=DEV)
    up = torch.as_tensor(rng.normal(0, 1, (60, 40)), dtype=torch.float32, device=DEV)
    up[n:] = 0
    left = float((nq.moe_gather(x, plan).double() * up.double()).sum())
    right = float((x.double() * nq.moe_combine(up, plan).double()).sum())
    assert abs(left - right) <= slack


def test_rows_strides_and_addresses():
    rng = np.random.default_rng(4)
    ids = choices(rng, 30, 4, 9, "half")
    plan = plan_of(ids, 9)
    base = torch.as_tensor(rng.normal(0, 1, (120, 300)), dtype=torch.bfloat16, device=DEV)
    w = torch.as_tensor(rng.random((30, 4)), dtype=torch.float32, device=DEV)
    for lo, hi in ((8, 264), (3, 259), (1, 100), (0, 300)):
        part, grad = base[:, lo:hi], base[:30, lo:hi]
        assert torch.equal(nq.moe_gather(base[:30, lo:hi], plan), nq.moe_gather(base[:30, lo:hi].contiguous(), plan))
        assert torch.equal(nq.moe_combine(part, plan, w), nq.moe_combine(part.contiguous(), plan, w))
        a, b = nq.moe_combine_grad(grad, part, plan, w), nq.moe_combine_grad(grad.contiguous(), part.contiguous(), plan, w)
        assert torch.equal(a[0], b[0]) and torch.allclose(a[1], b[1], rtol=0, atol=300 * 25 * 2.0 ** -23)
    one = base[:1, :256].expand(30, 256)  # a gradient that is one row for all tokens
    a, b = nq.moe_combine_grad(one, base[:, :256], plan, w), nq.moe_combine_grad(one.contiguous(), base[:, :256], plan, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --- the experts' products --------------------------------------------------------------------------------------

def experts_run(rng, tokens, top, experts, n, k, kind, sorted_rows, gated, dtype, out, codes):
    ids = choices(rng, tokens, top, experts, kind)
    plan = plan_of(ids, experts)
    order, _, offsets = fp8_ref.sort(ids, experts)
    x = values(rng, tokens * top if sorted_rows else tokens, k, dtype, 0.5)
    ww, ws = weight(rng, experts, n, k)
    announce(f"moe_gemm_fp8_block {tokens} x {top} of {experts} [{n}, {k}] {kind} sorted {sorted_rows} gated {gated} {dtype} -> {out} codes {codes}")
    xd = x.to(DEV)
    xs = None
    if codes:
        xd, xs = nq.quantize_fp8_block(xd)
    y = nq.moe_gemm_fp8_block(handle(ww, ws), xd, plan, xs, sorted_rows, gated, DT[out])
    torch.cuda.synchronize()
    wide = out == "f32" or fp8_ref.few_rows(tokens * top, experts)
    want = fp8_ref.experts_product(*fp8_ref.quantize(x.float().numpy()), ww, ws, order, offsets, top, sorted_rows, wide, gated)
    fp8_ref.check(y, *want, f"experts {kind}")
    assert not bool(y[int(offsets[-1]):].any())


@pytest.mark.parametrize("tokens, top, experts", [(1, 1, 1), (1, 4, 8), (5, 2, 60), (40, 4, 8), (120, 6, 12), (300, 2, 5), (700, 1, 2)])
@pytest.mark.parametrize("kind", ["random", "one", "few", "half", "none"])
def test_experts(tokens, top, experts, kind):
    rng = np.random.default_rng(tokens)
    gated = tokens % 2 == 0
    experts_run(rng, tokens, top, experts, 256 if gated else 70, 256, kind, kind in ("few", "half"), gated,
                ("bf16", "f32", "f16")[tokens % 3], ("bf16", "f32")[top % 2], kind == "random")


@pytest.mark.parametrize("sorted_rows", [False, True])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("tokens", [3, 50, 200])
def test_experts_forms(tokens, out, sorted_rows):
    rng = np.random.default_rng(tokens)
    for codes in (False, True):
        experts_run(rng, tokens, 3, 4, 130, 640, "half", sorted_rows, False, "f16", out, codes)
        experts_run(rng, tokens, 3, 4, 512, 128, "random", sorted_rows, True, "bf16", out, codes)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_experts_odd_widths(out):
    """Rows that begin at any element, many of them behind the last place."""
    experts_run(np.random.default_rng(3), 300, 4, 12, 1027, 128, "half", False, False, "bf16", out, False)


def test_many_experts():
    experts_run(np.random.default_rng(1), 70, 8, 1024, 20, 128, "random", False, False, "bf16", "bf16", False)


def test_experts_largest_tiles():
    rng = np.random.default_rng(2)
    experts_run(rng, 2100, 2, 4, 256, 128, "random", False, True, "bf16", "bf16", False)
    tokens, top, experts, n, k = 6000, 4, 12, 4096, 128
    ids = choices(rng, tokens, top, experts)
    plan, (order, _, offsets) = plan_of(ids, experts), fp8_ref.sort(ids, experts)
    x = values(rng, tokens, k, "bf16", 0.5)
    ww, ws = weight(rng, experts, n, k)
    y = nq.moe_gemm_fp8_block(handle(ww, ws), x.to(DEV), plan)
    xw, xs = fp8_ref.quantize(x.float().numpy())
    for p in np.unique(np.r_[offsets[:-1], offsets[1:] - 1, rng.integers(0, tokens * top, 30)]):
        e = np.searchsorted(offsets, p, side="right") - 1
        r = order[p:p + 1] // top
        want = fp8_ref.product(xw[r], xs[r], ww[e], ws[e], False)
        fp8_ref.check(y[p:p + 1], *want, f"place {p}")


@pytest.mark.parametrize("tokens", [6, 90, 400])
def test_plan_of_any_words_stays_inside(tokens):
    """Orders, places and offsets that no sort gives: nothing outside the tensors is read or written."""
    rng = np.random.default_rng(tokens)
    top, experts, n, k = 2, 5, 256, 128
    any32 = lambda *s: torch.as_tensor(rng.choice([-2 ** 31, -7, 0, 3, tokens, 2 * tokens - 1, 2 * tokens, 2 ** 31 - 1], s),  # noqa: E731
                                       dtype=torch.int32, device=DEV)
    ww, ws = weight(rng, experts, n, k)
    w = handle(ww, ws)
    x = values(rng, tokens, k, "bf16").to(DEV)
    rows = values(rng, tokens * top, k, "bf16").to(DEV)
    for i in range(3):
        plan = nq.MoePlan(any32(tokens * top), any32(tokens, top), any32(experts + 1))
        announce(f"any plan {tokens} {i}")
        nq.moe_gemm_fp8_block(w, x, plan)
        nq.moe_gemm_fp8_block(w, rows, plan, sorted_rows=True, gated=True)
        nq.moe_gather(x, plan)
        nq.moe_combine(rows, plan)
        nq.moe_combine_grad(x, rows, plan, torch.ones((tokens, top), device=DEV))
        torch.cuda.synchronize()


# --- together ---------------------------------------------------------------------------------------------------

def layer(x, ids, weights, w13, w2):
    plan = nq.moe_sort(ids, w13.experts)
    h = nq.moe_gemm_fp8_block(w13, x, plan, gated=True)
    y = nq.moe_gemm_fp8_block(w2, h, plan, sorted_rows=True)
    return plan, h, y, nq.moe_combine(y, plan, weights)


@pytest.mark.parametrize("tokens", [1, 8, 100, 600])
def test_layer_of_experts(tokens):
    """Sort, gate and up, down, combine: each step against the formula on what the step before gave."""
    rng = np.random.default_rng(tokens)
    experts, top, hidden, inner = 8, 3, 256, 384
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)]).astype(np.int64)
    w1, s1 = weight(rng, experts, 2 * inner, hidden)
    w2, s2 = weight(rng, experts, hidden, inner)
    x = values(rng, tokens, hidden, "bf16", 0.3)
    w = rng.random((tokens, top)).astype(np.float32)
    announce(f"layer of experts {tokens}")
    a, b = handle(w1, s1), handle(w2, s2)
    plan, h, y, out = layer(x.to(DEV), torch.as_tensor(ids, device=DEV), torch.as_tensor(w, device=DEV), a, b)
    order, places, offsets = fp8_ref.sort(ids, experts)
    same_plan(plan, ids, experts, "layer")
    few = fp8_ref.few_rows(tokens * top, experts)
    q = lambda t: fp8_ref.quantize(t.float().cpu().numpy())  # noqa: E731
    fp8_ref.check(h, *fp8_ref.experts_product(*q(x), w1, s1, order, offsets, top, False, few, True), "gate and up")
    fp8_ref.check(y, *fp8_ref.experts_product(*q(h), w2, s2, order, offsets, top, True, few, False), "down")
    fp8_ref.check(out, *fp8_ref.combine(y.double().cpu().numpy(), places, w.astype(np.float64)), "combine")


@pytest.mark.parametrize("tokens", [4, 300])
def test_layer_in_a_graph(tokens):
    """Captured with one routing, replayed with others, the program's own work between the replays."""
    rng = np.random.default_rng(tokens)
    experts, top, hidden, inner = 16, 4, 256, 256
    a, b = handle(*weight(rng, experts, 2 * inner, hidden)), handle(*weight(rng, experts, hidden, inner))
    x = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((tokens, top), dtype=torch.int32, device=DEV)
    w = torch.zeros((tokens, top), device=DEV)
    layer(x, ids, w, a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(x, ids, w, a, b)
    for i in range(4):
        x.copy_(values(rng, tokens, hidden, "bf16", 0.3))
        ids.copy_(torch.as_tensor(choices(rng, tokens, top, experts, ("random", "half", "one", "few")[i])))
        w.copy_(torch.as_tensor(rng.random((tokens, top))))
        eager = layer(x, ids, w, a, b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0].order, eager[0].order) and torch.equal(captured[0].offsets, eager[0].offsets)
        for k in (1, 2, 3):
            assert torch.equal(captured[k], eager[k]), f"replay {i}, step {k}"


@pytest.mark.parametrize("tokens", [5, 64])
def test_example(tokens):
    """The example runs; its outputs are bfloat16: two roundings of 2^-8 of a value, and the sums' (fp8_ref.product)."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import experts_layer
    worst, gradient = experts_layer.main(tokens, 2)
    assert worst < 4 * 2.0 ** -8 and gradient < 1024 * 2.0 ** -23


def test_refusals():
    rng = np.random.default_rng(0)
    plan = plan_of(choices(rng, 6, 2, 4), 4)
    w = handle(*weight(rng, 4, 64, 128))
    one = handle(*weight(rng, 64, 128))
    x = torch.zeros((6, 128), device=DEV)
    for bad in (lambda: nq.moe_gemm_fp8_block(one, x, plan), lambda: nq.gemm_fp8_block(w, x),
                lambda: nq.moe_gemm_fp8_block(w, x, plan, sorted_rows=True), lambda: nq.moe_gemm_fp8_block(w, x[:5], plan),
                lambda: nq.moe_gemm_fp8_block(w, x, plan_of(choices(rng, 6, 2, 5), 5)),
                lambda: nq.moe_sort(torch.zeros(4, dtype=torch.int32, device=DEV), 4),
                lambda: nq.moe_sort(torch.zeros((4, 1), device=DEV), 4), lambda: nq.moe_sort(plan.places, 0),
                lambda: nq.moe_sort(plan.places, 1025), lambda: nq.moe_gather(x[:5], plan), lambda: nq.moe_combine(x, plan),
                lambda: nq.moe_combine(torch.zeros((12, 8), device=DEV), plan, torch.zeros((6, 3), device=DEV)),
                lambda: nq.moe_combine_grad(x, torch.zeros((12, 128), dtype=torch.bfloat16, device=DEV), plan),
                lambda: nq.MoePlan(plan.order[:5], plan.places, plan.offsets), lambda: nq.MoePlan(plan.order.long(), plan.places, plan.offsets)):
        with pytest.raises(ValueError):
            bad()
