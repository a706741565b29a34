"""Cases of the 8-bit key/value cache operators, to measure them and to compare them with their plain form.

Four operators of one serving step, over a pool of blocks of `block` tokens (codes of 8 bits, one binary32 scale for
each block and head; keys [blocks, heads, block, dim], values [blocks, heads, dim, block]):

* tables: block tables, slot map and token starts of a step from the requests' lengths (blocks come from a ring of
  free ones, finished requests give theirs back);
* store: new keys and values are quantized into their blocks;
* load: whole blocks come back as values;
* attention: queries of any number of tokens a request against the keys and values of their block table.

With `own` false, run() computes them in elementary torch operations; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
QMAX = {"q8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -126  # least scale


# --- cases ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of a small batch: one token each, now and then a new block, one request ends
        dict(name="tables decode 48", op="tables", requests=48, longest=4096, new=1, chunks=0, ends=1, block=64),
        # a full server's step: 1000 requests, some of them prompts of up to 4096 tokens, short blocks
        dict(name="tables mixed 1000", op="tables", requests=1000, longest=16384, new=4096, chunks=24, ends=40, block=16),
        # the new token of each of 64 requests, mostly into half filled blocks
        dict(name="store decode 64 q8", op="store", requests=64, longest=4096, new=1, heads=8, dim=128, block=64,
             code="q8", dtype="bf16", out="bf16"),
        # prompts of ragged lengths, about 16000 tokens together, in binary16
        dict(name="store prompts e4m3", op="store", requests=6, longest=1000, new=3500, heads=8, dim=128, block=32,
             code="e4m3", dtype="f16", out="bf16"),
        # one short conversation's context as values
        dict(name="load 23 blocks q8", op="load", blocks=23, heads=8, dim=128, block=64, code="q8", out="f32"),
        # a long context moved out of the cache
        dict(name="load 4099 blocks e4m3", op="load", blocks=4099, heads=8, dim=64, block=32, code="e4m3", out="bf16"),
        # one request's first tokens: latency alone
        dict(name="attention single 37", op="attention", requests=1, longest=37, shortest=37, new=1, q_heads=32,
             heads=8, dim=128, block=64, code="q8", dtype="bf16", window=0),
        # a serving batch's decode step, ragged lengths
        dict(name="attention decode 128", op="attention", requests=128, longest=8200, shortest=1, new=1, q_heads=32,
             heads=8, dim=128, block=64, code="q8", dtype="bf16", window=0),
        # two very long contexts, where only the split over keys fills the card
        dict(name="attention decode long", op="attention", requests=2, longest=131001, shortest=65537, new=1,
             q_heads=32, heads=8, dim=128, block=128, code="e4m3", dtype="f16", window=0),
        # drafted tokens verified, a key head for each query head, a sliding window, short blocks, binary32
        dict(name="attention verify f32", op="attention", requests=32, longest=5000, shortest=100, new=5, q_heads=16,
             heads=16, dim=64, block=16, code="q8", dtype="f32", window=2049),
        # a chunked-prefill step: prompts of up to 1100 tokens and single tokens together
        dict(name="attention mixed e4m3", op="attention", requests=24, longest=4100, shortest=1, new=1100, q_heads=32,
             heads=8, dim=128, block=32, code="e4m3", dtype="bf16", window=0),
        # the second half of a long prompt
        dict(name="attention prompt 4096", op="attention", requests=1, longest=8192, shortest=8192, new=4096,
             q_heads=32, heads=8, dim=128, block=64, code="q8", dtype="bf16", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "store", "load", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 64, 128])
    code = rng.choice(["q8", "e4m3"])
    heads, dim = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([64, 128, 128, 256])
    if op == "tables":
        b = _log(rng, 1, 1000)
        return dict(op=op, requests=b, longest=_log(rng, 64, 16384), new=rng.choice([1, 1, 3, _log(rng, 16, 4096)]),
                    chunks=rng.randint(0, min(b, 24)), ends=rng.randint(0, b // 8), block=block)
    if op == "store":
        while True:
            b, new = _log(rng, 1, 256), rng.choice([1, 2, _log(rng, 4, 4000)])
            if b * new * heads * dim <= 16000 * 8 * 128:
                return dict(op=op, requests=b, longest=_log(rng, 16, 4096), new=new, heads=heads, dim=dim, block=block,
                            code=code, dtype=rng.choice(list(DTYPES)), out=rng.choice(list(DTYPES)))
    if op == "load":
        n = _log(rng, 1, max(2, 4099 * 32 * 8 * 64 // (block * heads * dim)))
        return dict(op=op, blocks=n, heads=heads, dim=dim, block=block, code=code, out=rng.choice(list(DTYPES)))
    while True:
        b, new = _log(rng, 1, 128), rng.choice([1, 1, 1, 4, _log(rng, 2, 64), _log(rng, 64, 4096)])
        longest = max(new, _log(rng, 16, 131072))
        group = rng.choice([1, 2, 4, 4, 5, 8, 16])
        padded = b * heads * longest * dim  # values of the plain form's padded keys; its score count below
        if padded <= 128 * 8 * 8200 * 128 and b * heads * group * new * longest <= 32 * 4096 * 8192:
            return dict(op=op, requests=b, longest=longest, shortest=rng.choice([1, longest // 2 + 1]), new=new,
                        q_heads=heads * group, heads=heads, dim=dim, block=block, code=code,
                        dtype=rng.choice(list(DTYPES)), window=rng.choice([0, 0, 0, _log(rng, 1, longest)]))


# --- inputs -----------------------------------------------------------------------------------------------------

def _seed(seed):
    return np.random.default_rng(seed), torch.Generator(device=DEV).manual_seed(seed)


def _codes(shape, code, gen):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16)
    if code == "q8":
        return (x * 35).round_().clamp_(-127, 127).to(torch.int8)
    return (x * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _cache(c, blocks, gen):
    """A pool of earlier tokens: scales of a layer's keys and values (amax near 4) that differ from block to block."""
    h, d, t, code = c["heads"], c["dim"], c["block"], c["code"]
    scale = lambda: torch.exp(0.4 * torch.randn((blocks, h), generator=gen, device=DEV)) * 4.0 / QMAX[code]  # noqa: E731
    return dict(k=_codes((blocks, h, t, d), code, gen), v=_codes((blocks, h, d, t), code, gen), ks=scale(), vs=scale())


def _new_values(n, h, d, dtype, gen):
    """Keys or values of n tokens: normal, some channels ten times larger, rows of different size."""
    x = torch.randn((n, h, d), generator=gen, device=DEV)
    x[:, :, ::17] *= 6
    x *= torch.exp(0.5 * torch.randn((n, h, 1), generator=gen, device=DEV))
    return x.to(DTYPES[dtype])


def _lengths(c, order=None):
    """Each request's tokens in the cache before the step and its new ones, on the host: the case's own lengths, so
    that outputs have one shape, in an order of the seed's."""
    past, new = _case_lengths(c, np.random.default_rng(c["requests"]))
    order = np.arange(past.size) if order is None else order.permutation(past.size)
    return past[order], new[order]


def _case_lengths(c, np_rng):
    b = c["requests"]
    if c["op"] == "attention":
        total = np.exp(np_rng.uniform(math.log(c["shortest"]), math.log(c["longest"]), b)).astype(np.int64)
        total = np.clip(total, c["shortest"], c["longest"])
        total[0] = c["longest"]
        new = np.full(b, c["new"])
        if c["new"] > 16 and b > 1:  # a chunked-prefill step: every third request has a chunk, the others one token
            new = np.where(np.arange(b) % 3 == 0, np_rng.integers(c["new"] // 2, c["new"] + 1, b), 1)
            new[0] = c["new"]
        new = np.minimum(new, total)
        return total - new, new
    past = np_rng.integers(0, c["longest"] + 1, b)
    if c["op"] == "tables":
        new = np.full(b, min(c["new"], 3))
        at = np_rng.permutation(b)[: c["chunks"]]
        new[at] = np_rng.integers(1, c["new"] + 1, at.size)
        new[np_rng.permutation(b)[: c["ends"]]] = -1
        return past, new
    new = np_rng.integers((c["new"] + 1) // 2, c["new"] + 1, b) if c["new"] > 2 else np.full(b, c["new"])
    return past, new


def _host_tables(past, new, block, np_rng, spare):
    """Block table, slots and token starts of requests that already hold their blocks, from a shuffled pool."""
    total = past + new
    need = -(-total // block)
    blocks = int(need.sum()) + spare
    order = np_rng.permutation(blocks)
    first = np.concatenate([[0], np.cumsum(need)])
    width = max(1, int(need.max()))
    col = np.arange(width)
    table = np.where(col < need[:, None], order[np.minimum(first[:-1, None] + col, blocks - 1)], -1)
    starts = np.concatenate([[0], np.cumsum(new)])
    b = np.repeat(np.arange(past.size), new)
    pos = past[b] + np.arange(starts[-1]) - starts[b]
    slots = table[b, pos // block] * block + pos % block
    touched = np.unique(slots // block)
    return table, slots, starts, touched, blocks


def _gpu(x, dtype):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype, device=DEV)


def prepare(case, seed):
    c = case
    np_rng, gen = _seed(seed)
    s = dict(c=c)
    if c["op"] == "tables":
        past, new = _lengths(c, np_rng)
        held = -(-past // c["block"])
        want = np.where(new > 0, -(-(past + new) // c["block"]) - held, 0)
        blocks = int(held.sum() + want.sum()) + 64
        order = np_rng.permutation(blocks)
        width = int((held + want).max()) + 2
        first = np.concatenate([[0], np.cumsum(held)])
        col = np.arange(width)
        table = np.where(col < held[:, None], order[np.minimum(first[:-1, None] + col, blocks - 1)], -1)
        head, count = int(np_rng.integers(0, blocks)), blocks - int(held.sum())
        ring = np.full(blocks, -1)
        ring[(head + np.arange(count)) % blocks] = order[blocks - count:]
        s.update(lengths=_gpu(past, torch.int32), new=_gpu(new, torch.int32), table=_gpu(table, torch.int32),
                 ring=_gpu(ring, torch.int32), state=_gpu([head, count], torch.int32),
                 tokens=int(np.maximum(new, 0).sum()) + 7)
        return s
    if c["op"] == "load":
        pool = c["blocks"] + 5
        s.update(cache=_cache(c, pool, gen), ids=_gpu(np_rng.permutation(pool)[: c["blocks"]], torch.int32))
    else:
        past, new = _lengths(c, np_rng)
        table, slots, starts, touched, blocks = _host_tables(past, new, c["block"], np_rng, 3)
        s.update(cache=_cache(c, blocks, gen), starts=_gpu(starts, torch.int32), lengths=_gpu(past + new, torch.int32),
                 table=_gpu(table, torch.int32))
        n = int(starts[-1])
        if c["op"] == "store":
            s.update(k=_new_values(n, c["heads"], c["dim"], c["dtype"], gen),
                     v=_new_values(n, c["heads"], c["dim"], c["dtype"], gen), slots=_gpu(slots, torch.int64),
                     ids=_gpu(touched, torch.int32))
        else:
            q = torch.randn((n, c["q_heads"], c["dim"]), generator=gen, device=DEV)
            s.update(q=q.to(DTYPES[c["dtype"]]), max_new=int(new.max()), max_length=int((past + new).max()),
                     scale=1.0 / math.sqrt(c["dim"]))
    if own:
        import block_quantized_weight_nq_amd as nq
        k = s["cache"]
        s["handle"] = nq.KvCache(k["k"], k["v"], k["ks"], k["vs"])
    return s


# --- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["c"]["op"]](state)


def _own_tables(s):
    import block_quantized_weight_nq_amd as nq
    t = nq.kv_tables(s["lengths"], s["new"], s["table"], s["ring"], s["state"], s["c"]["block"], s["tokens"])
    return dict(table=s["table"], ring=s["ring"], lengths=t.lengths, starts=t.token_start, slots=t.slots,
                state=t.free_state, status=t.status)


def _own_store(s):
    import block_quantized_weight_nq_amd as nq
    status = nq.kv_store(s["handle"], s["k"], s["v"], s["slots"], s["starts"])
    k, v = nq.kv_load(s["handle"], s["ids"], DTYPES[s["c"]["out"]])
    return dict(k=k, v=v, ks=s["cache"]["ks"], vs=s["cache"]["vs"], status=status)


def _own_load(s):
    import block_quantized_weight_nq_amd as nq
    k, v = nq.kv_load(s["handle"], s["ids"], DTYPES[s["c"]["out"]])
    return dict(k=k, v=v)


def _own_attention(s):
    import block_quantized_weight_nq_amd as nq
    out, lse = nq.kv_attention(s["handle"], s["q"], s["starts"], s["lengths"], s["table"], scale=s["scale"],
                               window=s["c"]["window"], max_new=s["max_new"], max_length=s["max_length"],
                               return_lse=True)
    return dict(out=out, lse=lse)


def _plain_tables(s):
    block, n_tok, ring, table = s["c"]["block"], s["tokens"], s["ring"].long(), s["table"].long()
    length, new, (head, count) = s["lengths"].long(), s["new"].long(), s["state"].long().unbind()
    blocks, width = ring.numel(), table.shape[1]
    add, held = new.clamp(min=0), (length + block - 1) // block
    after = (length + add + block - 1) // block
    give = torch.where(new < 0, held, 0)
    need = after - held
    starts = torch.nn.functional.pad(add.cumsum(0), (1, 0))
    took, gave = need.cumsum(0), give.cumsum(0)
    status = torch.where(took[-1] > count, 1, 0)
    status = status | torch.where(((length < 0) | (new < -1) | (length + add > width * block)).any(), 2, 0)
    status = status | torch.where(starts[-1] > n_tok, 4, 0)
    status = status | torch.where((count < 0) | (head < 0) | (head >= blocks) | (count - took[-1] + gave[-1] > blocks), 8, 0)
    ok = status == 0
    col = torch.arange(width, device=DEV)
    fresh = ok & (col >= held[:, None]) & (col < after[:, None])
    at = (head + (took - need)[:, None] + col - held[:, None]) % blocks
    table = torch.where(fresh, ring[at], table)
    back = ok & (col < give[:, None])
    at = torch.where(back, (head + count + (gave - give)[:, None] + col) % blocks, blocks)
    ring = torch.nn.functional.pad(ring, (0, 1)).scatter(0, at.reshape(-1), table.reshape(-1))[:blocks]
    starts = torch.where(ok, starts, 0)
    i = torch.arange(n_tok, device=DEV)
    b = torch.searchsorted(starts[1:].contiguous(), i, right=True)
    live = b < length.numel()
    b = b.clamp(max=length.numel() - 1)
    pos = length[b] + i - starts[b]
    slots = torch.where(live, table[b, (pos // block).clamp(max=width - 1)] * block + pos % block, -1)
    out = torch.where(ok, torch.where(new < 0, 0, length + add), length)
    state = torch.where(ok, torch.stack([(head + took[-1]) % blocks, count - took[-1] + gave[-1]]), s["state"].long())
    as32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(table=as32(table), ring=as32(ring), lengths=as32(out), starts=as32(starts), slots=slots,
                state=as32(state), status=as32(status).reshape(1))


def _round_code(x, code):
    if code == "q8":
        return x.round().clamp(-127, 127)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _plain_store_one(s, x, codes, scales, tokens_last):
    """x [n, heads, dim] into codes; tokens_last: codes are [blocks, heads, dim, block]."""
    c, ids = s["c"], s["ids"].long()
    block, code = c["block"], c["code"]
    qmax = torch.full((1,), QMAX[code], device=DEV)
    page, off = s["slots"] // block, s["slots"] % block
    x = x.float()
    finite = x.isfinite()
    amax = torch.where(finite, x.abs(), 0).amax(-1)
    big = torch.zeros_like(scales).scatter_reduce(0, page[:, None].expand(-1, c["heads"]), amax, "amax")[ids]
    first = torch.full((scales.shape[0],), block, device=DEV).scatter_reduce(0, page, off, "amin")[ids]
    old = torch.where((first > 0)[:, None], scales[ids], 0)
    new = torch.maximum(old, (big / qmax).clamp(min=TINY))
    at = torch.arange(block, device=DEV)
    keep = (at < first[:, None])[:, None, :, None] & (new > old)[:, :, None, None]
    was = codes[ids].float()
    was = was.transpose(2, 3) if tokens_last else was
    now = torch.where(keep, _round_code(was * (old / new)[:, :, None, None], code), was)
    where = torch.searchsorted(ids, page)
    one = torch.ones(1, device=DEV)
    fresh = torch.where(x.isnan(), 0, x) * (one / new)[where][:, :, None]
    now.transpose(1, 2)[where, off] = _round_code(fresh, code)
    codes[ids] = (now.transpose(2, 3) if tokens_last else now).to(codes.dtype)
    scales[ids] = new
    return torch.where(finite.all(), 0, 1)


def _values(codes, scales, ids, tokens_last, out):
    ids = ids.long()
    x = codes[ids].float() * scales[ids][:, :, None, None]
    return (x.permute(0, 3, 1, 2) if tokens_last else x.transpose(1, 2)).to(DTYPES[out]).contiguous()


def _plain_load(s):
    k = s["cache"]
    return dict(k=_values(k["k"], k["ks"], s["ids"], False, s["c"]["out"]),
                v=_values(k["v"], k["vs"], s["ids"], True, s["c"]["out"]))


def _plain_store(s):
    k = s["cache"]
    bad = _plain_store_one(s, s["k"], k["k"], k["ks"], False) | _plain_store_one(s, s["v"], k["v"], k["vs"], True)
    return dict(_plain_load(s), ks=k["ks"], vs=k["vs"], status=bad.to(torch.int32).reshape(1))


def _plain_attention(s):
    c, k = s["c"], s["cache"]
    h, d, block, group, mn = c["heads"], c["dim"], c["block"], c["q_heads"] // c["heads"], s["max_new"]
    starts, lengths = s["starts"].long(), s["lengths"].long()
    b, nb = lengths.numel(), -(-s["max_length"] // block)
    ids = s["table"].long()[:, :nb].clamp(min=0)
    keys = k["k"][ids].float().mul_(k["ks"][ids][..., None, None]).permute(0, 2, 1, 3, 4).reshape(b, h, nb * block, d)
    values = k["v"][ids].float().mul_(k["vs"][ids][..., None, None]).permute(0, 2, 1, 4, 3).reshape(b, h, nb * block, d)
    j = torch.arange(mn, device=DEV)
    new = starts[1:] - starts[:-1]
    q = s["q"].float()[(starts[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)]  # [b, mn, q_heads, d]
    q = q.reshape(b, mn, h, group, d).permute(0, 2, 1, 3, 4).reshape(b, h, mn * group, d)
    score = torch.matmul(q, keys.transpose(2, 3).contiguous()).mul_(s["scale"]).view(b, h, mn, group, nb * block)
    at, pos = torch.arange(nb * block, device=DEV), (lengths - new)[:, None] + j
    seen = (at <= pos[..., None]) & (at < lengths[:, None, None])
    if c["window"]:
        seen &= at > pos[..., None] - c["window"]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top.isfinite(), top, 0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(b, h, mn * group, nb * block), values).view(b, h, mn, group, d)
    out = out / torch.where(total > 0, total, 1)
    lse = (top + total.log()).squeeze(-1)
    i = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(starts[1:].contiguous(), i, right=True).clamp(max=b - 1)
    t = i - starts[r]
    return dict(out=out[r, :, t].reshape(s["q"].shape).to(s["q"].dtype), lse=lse[r, :, t].reshape(s["q"].shape[:2]))


_own = dict(tables=_own_tables, store=_own_store, load=_own_load, attention=_own_attention)
_plain = dict(tables=_plain_tables, store=_plain_store, load=_plain_load, attention=_plain_attention)


# --- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "load":
        n = c["blocks"] * c["block"] * c["heads"] * c["dim"] * 2
        return dict(bytes=n * (1 + DTYPES[c["out"]].itemsize) + 8 * c["blocks"] * c["heads"], flops=n)
    past, new = _lengths(c)
    if c["op"] == "tables":
        t = c["block"]
        moved = np.where(new > 0, -(-(past + new) // t) - -(-past // t), np.where(new < 0, -(-past // t), 0))
        n = int(np.maximum(new, 0).sum())
        return dict(bytes=8 * (n + 7) + 8 * int(moved.sum()) + 16 * past.size, flops=4 * n)
    if c["op"] == "store":
        n = int(new.sum()) * c["heads"] * c["dim"] * 2
        touched = int((-(-(past + new) // c["block"]) - past // c["block"]).sum())
        held = touched * c["block"] * c["heads"] * c["dim"] * 2  # the blocks read back
        return dict(bytes=n * (DTYPES[c["dtype"]].itemsize + 1) + held * (1 + DTYPES[c["out"]].itemsize)
                    + 24 * touched * c["heads"], flops=4 * n + held)
    total = past + new
    w = c["window"] or int(total.max())
    first = np.maximum(0, past + 1 - w)  # the first query's first key
    kv = int((total - first).sum()) * c["heads"]
    pairs = 0
    for p, n in zip(past.tolist(), new.tolist()):
        pairs += int(np.minimum(np.arange(p + 1, p + n + 1), w).sum())
    rows = int(new.sum()) * c["q_heads"]
    size = DTYPES[c["dtype"]].itemsize
    return dict(bytes=kv * c["dim"] * 2 + 8 * kv // c["block"] + rows * (2 * c["dim"] * size + 4),
                flops=4 * pairs * c["q_heads"] * c["dim"])


# --- the definition in 64 bits ----------------------------------------------------------------------------------

def _e4m3(x):
    """The nearest E4M3 value (ties to even), at most 448."""
    x = np.clip(x, -448, 448)
    with np.errstate(divide="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.abs(x))), -6) - 3)
    return np.rint(x / step) * step


def _exact_store(s):
    """The definition names binary32 for the scale, its inverse and the value that becomes a code, so these are rounded
    to it here too: a code next to a border is what the definition says. The rest is in 64 bits."""
    c, one = s["c"], np.float32
    t, qmax = c["block"], QMAX[c["code"]]
    nearest = _e4m3 if c["code"] == "e4m3" else lambda y: np.clip(np.rint(y), -127, 127)
    slots, ids = s["slots"].cpu().numpy(), s["ids"].cpu().numpy()
    page = slots // t
    res = {}
    for name, tokens_last in (("k", False), ("v", True)):
        codes = s["cache"][name][s["ids"].long()].float().cpu().numpy().astype(np.float64)
        codes = codes.swapaxes(2, 3) if tokens_last else codes
        scales = s["cache"][name + "s"].cpu().numpy().copy()
        x = s[name].float().cpu().numpy()
        for n, block in enumerate(ids):
            rows = np.nonzero(page == block)[0]
            off = slots[rows] % t
            old = scales[block] if off[0] else np.zeros(c["heads"], one)
            new = np.maximum(old, np.maximum(np.abs(x[rows]).max((0, 2)) / one(qmax), one(TINY)))
            for h in np.nonzero(new > old)[0]:
                codes[n, h, : off[0]] = nearest((codes[n, h, : off[0]].astype(one) * (old[h] / new[h])).astype(np.float64))
            codes[n][:, off] = nearest((x[rows] * (one(1) / new)[:, None]).astype(np.float64)).swapaxes(0, 1)
            scales[block] = new
        res[name] = torch.from_numpy((codes * scales[ids][:, :, None, None].astype(np.float64)).swapaxes(1, 2).copy())
        res[name + "s"] = torch.from_numpy(scales.astype(np.float64))
    return dict(res, status=None)


def _exact_attention(s):
    c, k = s["c"], s["cache"]
    h, d, t, group = c["heads"], c["dim"], c["block"], c["q_heads"] // c["heads"]
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lengths):
        q0, q1 = starts[b], starts[b + 1]
        if q0 == q1:
            continue
        ids = s["table"][b, : -(-n // t)].long()
        for head in range(h):
            kk = (k["k"][ids, head].double() * k["ks"][ids, head].double()[:, None, None]).reshape(-1, d)[:n]
            vv = (k["v"][ids, head].double() * k["vs"][ids, head].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:n]
            for g in range(group):
                at = head * group + g
                p = torch.mm(s["q"][q0:q1, at].double(), kk.t().contiguous()) * s["scale"]
                pos = torch.arange(n - (q1 - q0), n, device=DEV)[:, None]
                key = torch.arange(n, device=DEV)[None]
                hidden = key > pos
                if c["window"]:
                    hidden |= key <= pos - c["window"]
                p = p.masked_fill(hidden, -math.inf)
                lse[q0:q1, at] = torch.logsumexp(p, 1)
                out[q0:q1, at] = torch.mm(torch.softmax(p, 1), vv)
    return dict(out=out, lse=lse)


def exact(case, seed):
    """What run() returns, in 64 bits; None for the tables, which are whole numbers."""
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(s)
    if case["op"] == "load":
        ids = s["ids"].long()
        value = lambda n: s["cache"][n][ids].double() * s["cache"][n + "s"][ids].double()[:, :, None, None]  # noqa: E731
        return dict(k=value("k").transpose(1, 2), v=value("v").permute(0, 3, 1, 2))
    return _exact_attention(s)
