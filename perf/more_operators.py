"""Cases of the 8-bit floating-point block operators and of the experts' routing, to measure them and to compare them
with their plain form.

E4M3 codes with one binary32 scale for each block of 128: activations have a scale for each row and 128 columns,
weights one for each tile of 128 rows by 128 columns. Five operators, which together are a layer of experts (and the
second alone a linear layer):

* quantize: values become codes and scales, and codes become values again;
* product: activations (rounded to codes within the call, or codes already) times a weight, with silu(gate) * up as
  an epilogue where the weight holds both;
* sort: the (token, choice) pairs of a router in the experts' order, and the tokens' rows in it;
* experts: each expert's weight times the rows that are its own;
* combine: the experts' rows back to their tokens, weighted and summed, and the gradients of that.

With `own` false, run() computes them in elementary torch operations; with `own` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOP = 448.0  # largest E4M3 value
TINY = 2.0 ** -126  # least scale
B = 128


# --- cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the activations of a decode step of seven requests: latency alone
        dict(name="quantize 7 rows", op="quantize", rows=7, cols=4096, tile=1, dtype="bf16", back=""),
        # a projection's weight when a model is loaded, and its values again
        dict(name="quantize weight", op="quantize", rows=14336, cols=4096, tile=128, dtype="bf16", back="bf16"),
        # gate and up projection of one token
        dict(name="product decode 1", op="product", m=1, n=28672, k=4096, gated=True, dtype="bf16", codes=False, out="bf16"),
        # down projection of a batch's odd number of tokens, in binary16
        dict(name="product 77", op="product", m=77, n=4096, k=14336, gated=False, dtype="f16", codes=False, out="f16"),
        # gate and up projection of a long prompt
        dict(name="product prompt 8192", op="product", m=8192, n=28672, k=4096, gated=True, dtype="bf16", codes=False, out="bf16"),
        # the router's choices of a decode step
        dict(name="sort decode 5", op="sort", tokens=5, top=8, experts=64, among=64, cols=0, dtype="bf16"),
        # those of many prompts, and the tokens' rows in the experts' order
        dict(name="sort prompts 16384", op="sort", tokens=16384, top=8, experts=256, among=256, cols=2048, dtype="bf16"),
        # gate and up projections of four requests' tokens: a few rows for each of some thirty experts
        dict(name="experts decode 4", op="experts", tokens=4, top=8, experts=64, among=64, n=2816, k=2048, gated=True, sorted=False,
             dtype="bf16", codes=False, out="bf16"),
        # down projections of a ragged batch on a device that holds half of the experts
        dict(name="experts 300 of half", op="experts", tokens=300, top=6, experts=64, among=128, n=2048, k=1408, gated=False, sorted=True,
             dtype="f16", codes=False, out="f16"),
        # gate and up projections of long prompts
        dict(name="experts prompts 8192", op="experts", tokens=8192, top=8, experts=64, among=64, n=2816, k=2048, gated=True, sorted=False,
             dtype="bf16", codes=False, out="bf16"),
        # the experts' rows of a decode step back to their tokens
        dict(name="combine decode 5", op="combine", tokens=5, top=8, experts=64, among=64, cols=2048, dtype="bf16", grad=False),
        # those of a training step over a router, with the gradients of rows and weights
        dict(name="combine train 8192", op="combine", tokens=8192, top=8, experts=64, among=64, cols=2048, dtype="bf16", grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "sort", "experts", "experts", "combine"])
    dtype = rng.choice(list(DTYPES))
    if op == "quantize":
        tile = rng.choice([1, 1, 128])
        cols = B * _log(rng, 1, 128)
        return dict(op=op, rows=_log(rng, 1, max(1, 14336 * 4096 // cols // (2 if dtype == "f32" else 1))), cols=cols, tile=tile,
                    dtype=dtype, back=rng.choice(["", *DTYPES]))
    tokens, top = _log(rng, 1, 16384), rng.choice([1, 2, 4, 6, 8])
    experts = max(top, rng.choice([4, 8, 16, 60, 64, 128, 256]))
    routed = dict(tokens=tokens, top=top, experts=experts, among=experts * rng.choice([1, 1, 1, 2, 4]))
    if op == "sort":
        return dict(op=op, **routed, cols=rng.choice([0, 8 * _log(rng, 8, 256)]), dtype=rng.choice(["f16", "bf16"]))
    if op == "combine":
        cols = min(8 * _log(rng, 8, 1024), 8 * (8192 * 2048 // tokens // (2 if dtype == "f32" else 1) // top))
        return dict(op=op, **routed, cols=max(8, cols), dtype=dtype, grad=rng.choice([False, True]))
    gated = rng.choice([False, True])
    form = dict(gated=gated, dtype=dtype, codes=rng.choice([False, False, True]), out=rng.choice(["bf16", dtype]))
    if op == "product":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 32, 28672), B * _log(rng, 1, 128)
            n = max(2 * B, n // (2 * B) * 2 * B) if gated else n
            if m * n * k <= 8192 * 28672 * 4096 and n * k <= 28672 * 4096:
                return dict(op=op, m=m, n=n, k=k, **form)
    while True:
        n, k = _log(rng, 64, 8192), B * _log(rng, 1, 56)
        n = max(2 * B, n // (2 * B) * 2 * B) if gated else n
        tokens = _log(rng, 1, 8192)
        if tokens * top * n * k <= 8192 * 8 * 2816 * 2048 and experts * n * k <= 64 * 2816 * 2048:
            return dict(op=op, **{**routed, "tokens": tokens}, n=n, k=k, sorted=rng.choice([False, True]), **form)


# --- inputs -----------------------------------------------------------------------------------------------------

def _values(rows, cols, dtype, gen):
    """Activations: normal, some columns larger, rows of different size."""
    x = torch.randn((rows, cols), generator=gen, device=DEV)
    x[:, ::61] *= 6
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=DEV))
    return x.to(DTYPES[dtype])


def _weight(c, gen, experts=()):
    """Codes and scales of a weight of entries near 0.02 (or one for each expert)."""
    n, k = c["n"], c["k"]
    codes = torch.empty((*experts, n, k), dtype=torch.float8_e4m3fn, device=DEV)
    for part in codes.view(-1, n, k):  # one matrix at a time, so that the draws in 16 bits stay small
        part.copy_((torch.randn((n, k), generator=gen, device=DEV, dtype=torch.float16) * 100).clamp_(-TOP, TOP))
    scales = torch.exp(0.3 * torch.randn((*experts, -(-n // B), k // B), generator=gen, device=DEV)) * 2e-4
    return codes, scales


def _ids(c, gen):
    """A router's choices, [tokens, top] different experts a token, some experts preferred. Those from `experts` on
    are on another device."""
    taste = torch.randn((1, c["among"]), generator=gen, device=DEV) * 0.5
    score = torch.randn((c["tokens"], c["among"]), generator=gen, device=DEV) + taste
    return score.topk(c["top"], dim=1).indices.to(torch.int32)


def _routed(c, gen):
    """A plan that a program has in hand: the pairs in the experts' order."""
    ids = _ids(c, gen)
    order, places, offsets = _sort(ids, c["experts"])
    return dict(order=order, places=places, offsets=offsets, cap=max(1, int((offsets[1:] - offsets[:-1]).max())))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "quantize":
        s["x"] = _values(c["rows"], c["cols"], c["dtype"], gen)
        return s
    if c["op"] == "sort":
        s["ids"] = _ids(c, gen)
        if c["cols"]:
            s["x"] = _values(c["tokens"], c["cols"], c["dtype"], gen)
        return s
    if c["op"] == "product":
        s["w"], s["ws"] = _weight(c, gen)
        s["x"] = _values(c["m"], c["k"], c["dtype"], gen)
    else:
        s.update(_routed(c, gen))
        pairs = c["tokens"] * c["top"]
        if c["op"] == "combine":
            s["rows"] = _values(pairs, c["cols"], c["dtype"], gen)
            s["weights"] = torch.softmax(torch.randn((c["tokens"], c["top"]), generator=gen, device=DEV), 1)
            if c["grad"]:
                s["grad"] = _values(c["tokens"], c["cols"], c["dtype"], gen)
        else:
            s["w"], s["ws"] = _weight(c, gen, (c["experts"],))
            s["x"] = _values(pairs if c["sorted"] else c["tokens"], c["k"], c["dtype"], gen)
    if c.get("codes"):
        s["x"], s["xs"] = _quantize(s["x"], 1)
    if own:
        import block_quantized_weight_nq_amd as nq
        if "w" in s:
            s["handle"] = nq.Fp8Weight(s["w"], s["ws"])
        if "order" in s:
            s["plan"] = nq.MoePlan(s["order"], s["places"], s["offsets"])
    return s


# --- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["c"]["op"]](state)


def _own_quantize(s):
    import block_quantized_weight_nq_amd as nq
    c = s["c"]
    codes, scales = nq.quantize_fp8_block(s["x"], tile=c["tile"])
    if not c["back"]:
        return dict(codes=codes, scales=scales)
    return dict(values=nq.dequantize_fp8_block(codes, scales, tile=c["tile"], out_dtype=DTYPES[c["back"]]), scales=scales)


def _own_product(s):
    import block_quantized_weight_nq_amd as nq
    c = s["c"]
    return nq.gemm_fp8_block(s["handle"], s["x"], x_scales=s.get("xs"), gated=c["gated"], out_dtype=DTYPES[c["out"]])


def _own_sort(s):
    import block_quantized_weight_nq_amd as nq
    plan = nq.moe_sort(s["ids"], s["c"]["experts"])
    out = dict(order=plan.order, places=plan.places, offsets=plan.offsets)
    if "x" in s:
        out["rows"] = nq.moe_gather(s["x"], plan)
    return out


def _own_experts(s):
    import block_quantized_weight_nq_amd as nq
    c = s["c"]
    return nq.moe_gemm_fp8_block(s["handle"], s["x"], s["plan"], x_scales=s.get("xs"), sorted_rows=c["sorted"], gated=c["gated"],
                                 out_dtype=DTYPES[c["out"]])


def _own_combine(s):
    import block_quantized_weight_nq_amd as nq
    out = dict(out=nq.moe_combine(s["rows"], s["plan"], s["weights"]))
    if "grad" in s:
        out["grad_rows"], out["grad_weights"] = nq.moe_combine_grad(s["grad"], s["rows"], s["plan"], s["weights"])
    return out


def _blocks(x, tile):
    """[rows, cols] as [row tiles, tile, column blocks, 128], short tiles filled up with zeros."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, -rows % tile))
    return x.view(-1, tile, cols // B, B)


def _quantize(x, tile):
    """The scale is RN32(amax / 448), at least 2^-126, the code the nearest to RN32(x * RN32(1 / scale))."""
    rows, cols = x.shape
    x = _blocks(x.float(), tile)
    scales = (x.abs().amax((1, 3)) / torch.full((1,), TOP, device=DEV)).clamp(min=TINY)
    y = x * (torch.ones(1, device=DEV) / scales)[:, None, :, None]
    codes = y.clamp(-TOP, TOP).view(-1, cols)[:rows].to(torch.float8_e4m3fn)
    return codes, scales


def _dequantize(codes, scales, tile):
    rows, cols = codes.shape
    return (_blocks(codes.float(), tile) * scales[:, None, :, None]).view(-1, cols)[:rows]


def _activations(s):
    """The numbers that the products take for the activations, in 32 bits."""
    codes, scales = (s["x"], s["xs"]) if "xs" in s else _quantize(s["x"], 1)
    return _dequantize(codes, scales, 1)


def _finish(y, c):
    """y: [rows, n] sums in 32 bits."""
    if c["gated"]:
        gate, up = y[:, : c["n"] // 2], y[:, c["n"] // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(DTYPES[c["out"]])


def _plain_quantize(s):
    c = s["c"]
    codes, scales = _quantize(s["x"], c["tile"])
    if not c["back"]:
        return dict(codes=codes, scales=scales)
    return dict(values=_dequantize(codes, scales, c["tile"]).to(DTYPES[c["back"]]), scales=scales)


def _plain_product(s):
    w = _dequantize(s["w"], s["ws"], B)
    return _finish(torch.mm(_activations(s), w.t()), s["c"])


def _sort(ids, experts):
    """Pairs sorted by expert, in the order of tokens and choices within one; pairs of other experts are left out."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=DEV))
    at = torch.arange(flat.numel(), device=DEV)
    live = at < offsets[-1]
    places = torch.zeros_like(flat).scatter(0, order, torch.where(live, at, -1))
    order = torch.where(live, order, -1)
    return order.to(torch.int32), places.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def _plain_sort(s):
    order, places, offsets = _sort(s["ids"], s["c"]["experts"])
    out = dict(order=order, places=places, offsets=offsets)
    if "x" in s:
        token = order.long().clamp(min=0) // s["c"]["top"]
        out["rows"] = torch.where((order >= 0)[:, None], s["x"][token], 0)
    return out


def _plain_experts(s):
    c, order, offsets = s["c"], s["order"].long(), s["offsets"].long()
    x = _activations(s)
    if not c["sorted"]:
        x = x[order.clamp(min=0) // c["top"]]
    pairs, e, n, k = order.numel(), c["experts"], c["n"], c["k"]
    # each expert's rows, filled up to the most that one has; row `pairs` is the one of the places left over
    at = offsets[:-1, None] + torch.arange(s["cap"], device=DEV)
    at = torch.where(at < offsets[1:, None], at, pairs)
    x = torch.nn.functional.pad(x, (0, 0, 0, 1))[at.view(-1)].view(e, s["cap"], k)
    wide = torch.nn.functional.pad(s["w"].float(), (0, 0, 0, -n % B)).view(e, -1, B, k // B, B)
    w = (wide * s["ws"][:, :, None, :, None]).view(e, -1, k)[:, :n]
    y = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2).reshape(-1, n)
    out = torch.zeros((pairs + 1, n), device=DEV)
    out[at.view(-1)] = y
    out[pairs] = 0
    return _finish(out[:pairs], c)


def _plain_combine(s):
    c, places, w = s["c"], s["places"].long(), s["weights"]
    live = places >= 0
    rows = s["rows"].float()[places.clamp(min=0).view(-1)].view(*places.shape, -1)
    w = torch.where(live, w, 0)
    out = dict(out=(rows * w[..., None]).sum(1).to(s["rows"].dtype))
    if "grad" in s:
        grad = s["grad"].float()
        out["grad_weights"] = torch.where(live, (rows * grad[:, None]).sum(2), 0)
        order = s["order"].long()
        pair = order.clamp(min=0)
        g = grad[pair // c["top"]] * w.view(-1)[pair][:, None]
        out["grad_rows"] = torch.where((order >= 0)[:, None], g, 0).to(s["rows"].dtype)
    return out


_own = dict(quantize=_own_quantize, product=_own_product, sort=_own_sort, experts=_own_experts, combine=_own_combine)
_plain = dict(quantize=_plain_quantize, product=_plain_product, sort=_plain_sort, experts=_plain_experts, combine=_plain_combine)


# --- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    c = case
    size = lambda name: DTYPES[name].itemsize  # noqa: E731
    if c["op"] == "quantize":
        v = c["rows"] * c["cols"]
        scales = 4 * -(-c["rows"] // c["tile"]) * c["cols"] // B
        return dict(bytes=v * (size(c["dtype"]) + (size(c["back"]) if c["back"] else 1)) + scales, flops=v * (4 if c["back"] else 3))
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        x = m * k * (1 if c["codes"] else size(c["dtype"])) + (4 * m * k // B if c["codes"] else 0)
        return dict(bytes=n * k + 4 * -(-n // B) * k // B + x + m * n // (2 if c["gated"] else 1) * size(c["out"]), flops=2 * m * n * k)
    t, top = c["tokens"], c["top"]
    here = c["experts"] / c["among"]  # share of the pairs whose experts are here
    pairs = t * top * here
    if c["op"] == "sort":
        rows = (min(t, pairs) + t * top) * c["cols"] * size(c["dtype"])
        return dict(bytes=12 * t * top + 4 * c["experts"] + rows, flops=t * top)
    if c["op"] == "combine":
        h = c["cols"]
        both = c["grad"]
        return dict(bytes=(pairs + t * (2 if both else 1) + (t * top if both else 0)) * h * size(c["dtype"]) + t * top * (12 if both else 8),
                    flops=pairs * h * (5 if both else 2))
    n, k = c["n"], c["k"]
    busy = c["experts"] * (1 - (1 - top / c["among"]) ** t)  # experts that a token chose
    x = (pairs if c["sorted"] else min(t, pairs)) * k * (1 + 4 / B if c["codes"] else size(c["dtype"]))
    return dict(bytes=busy * (n * k + 4 * -(-n // B) * k // B) + x + t * top * (n // (2 if c["gated"] else 1) * size(c["out"]) + 4),
                flops=2 * pairs * n * k)


# --- the definition in 64 bits ----------------------------------------------------------------------------------
#
# The definition names binary32 for a scale, its inverse and the value that becomes a code, so these are rounded to it
# here too: a code next to a border is what the definition says. The rest is in 64 bits.

def _exact_codes(x, tile):
    """Codes and scales as numbers, a band of rows at a time."""
    rows, cols = x.shape
    codes, scales = torch.empty((rows, cols), dtype=torch.float32, device=DEV), []
    for r in range(0, rows, 2048):
        y = x[r:r + 2048].double()
        short = -y.shape[0] % tile
        y = torch.cat([y, y.new_zeros((short, cols))]).reshape(-1, tile, cols // B, B)
        scale = (y.abs().amax(3).amax(1) / TOP).float().clamp(min=TINY)
        scales.append(scale)
        y = (y * (1.0 / scale.double()).float().double()[:, None, :, None]).float().double().clamp(-TOP, TOP)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        y = torch.round(y / step) * step
        codes[r:r + 2048] = y.reshape(-1, cols)[: min(2048, rows - r)]
    return codes, torch.cat(scales)


def _exact_values(codes, scales, tile):
    wide = scales.double().repeat_interleave(tile, 0)[: codes.shape[0]].repeat_interleave(B, 1)
    return codes.double() * wide


def _exact_linear(x, w, ws, gated):
    y = torch.mm(x, _exact_values(w.float(), ws, B).t().contiguous())
    if gated:
        h = y.shape[1] // 2
        y = y[:, :h] * torch.sigmoid(y[:, :h]) * y[:, h:]
    return y


def exact(case, seed):
    """What run() returns, in 64 bits; None for whole numbers."""
    c = case
    s = prepare(case, seed)
    if c["op"] == "quantize":
        codes, scales = _exact_codes(s["x"], c["tile"])
        if not c["back"]:
            return dict(codes=codes.double(), scales=scales.double())
        return dict(values=_exact_values(codes, scales, c["tile"]), scales=scales.double())
    if c["op"] == "sort":
        if not c["cols"]:
            return None
        token = s["ids"].long().reshape(-1)
        token = torch.where((token < 0) | (token >= c["experts"]), c["experts"], token).argsort(stable=True)
        rows = s["x"].double()[token // c["top"]]
        n = int((s["ids"] < c["experts"]).sum())
        rows[n:] = 0
        return dict(order=None, places=None, offsets=None, rows=rows)
    if c["op"] == "combine":
        rows, w, grad = s["rows"].double(), s["weights"].double(), s["grad"].double() if "grad" in s else None
        out = torch.zeros((c["tokens"], c["cols"]), dtype=torch.float64, device=DEV)
        drows, dw = torch.zeros_like(rows), torch.zeros_like(w)
        for j in range(c["top"]):
            at = s["places"][:, j].long()
            t = torch.nonzero(at >= 0)[:, 0]
            out[t] += rows[at[t]] * w[t, j, None]
            if grad is not None:
                drows[at[t]] = grad[t] * w[t, j, None]
                dw[t, j] = (grad[t] * rows[at[t]]).sum(1)
        return dict(out=out) if grad is None else dict(out=out, grad_rows=drows, grad_weights=dw)
    if "xs" in s:
        x = _exact_values(s["x"].float(), s["xs"], 1)
    else:
        x = _exact_values(*_exact_codes(s["x"], 1), 1)
    if c["op"] == "product":
        return _exact_linear(x, s["w"], s["ws"], c["gated"])
    if not c["sorted"]:
        x = x[s["order"].long().clamp(min=0) // c["top"]]
    out = torch.zeros((x.shape[0], c["n"] // (2 if c["gated"] else 1)), dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    for e in range(c["experts"]):
        if ends[e] < ends[e + 1]:
            out[ends[e]:ends[e + 1]] = _exact_linear(x[ends[e]:ends[e + 1]], s["w"][e], s["ws"][e], c["gated"])
    return out
