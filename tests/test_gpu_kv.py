"""GPU: the 8-bit key/value cache operators against plain implementations (tests/kv_ref.py).

Tables, store and load are compared exactly: their definition fixes every rounding.  Attention is held to the error
bound of its arithmetic (kv_ref.check_attention).  Pools start with arbitrary words, NaN among the codes and scales of
what no token was stored in.
"""
import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import kv_ref
from gpu_util import announce
from kv_ref import CODE_DT, DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype, device=DEV)


def pool(rng, blocks, heads, block, dim, code, junk=True):
    """numpy codes (any word; E4M3 NaN among them) and scales of an arbitrary pool."""
    kc = rng.integers(0, 256, (blocks, heads, block, dim), dtype=np.uint8)
    vc = rng.integers(0, 256, (blocks, heads, dim, block), dtype=np.uint8)
    ks = np.exp(rng.normal(0, 1, (blocks, heads))).astype(np.float32) * 0.01
    vs = np.exp(rng.normal(0, 1, (blocks, heads))).astype(np.float32) * 0.01
    if not junk and code == "e4m3":
        kc[(kc & 127) == 127] ^= 1
        vc[(vc & 127) == 127] ^= 1
    if not junk and code == "q8":
        kc[kc == 128], vc[vc == 128] = 127, 127
    return kc, vc, ks, vs


def upload(kc, vc, ks, vs, code):
    k = dev(kc).view(CODE_DT[code])
    v = dev(vc).view(CODE_DT[code])
    return nq.KvCache(k, v, dev(ks), dev(vs))


def same_words(a, b, what):
    a = a.detach().cpu().view(torch.uint8).numpy()
    assert np.array_equal(a, b), f"{what}: {np.count_nonzero(a != b)} of {b.size} words differ"


# --- tables -----------------------------------------------------------------------------------------------------

def step(rng, R, longest, block, newest, ends, spare, extra):
    lengths = rng.integers(0, longest + 1, R).astype(np.int32)
    lengths[rng.integers(0, R, max(1, R // 5))] = rng.choice([0, block - 1, block, block + 1])
    added = rng.integers(0, newest + 1, R).astype(np.int32)
    added[rng.permutation(R)[:ends]] = -1
    held = -(-lengths // block)
    need = np.where(added > 0, -(-(lengths + added) // block) - held, 0)
    blocks = int(held.sum() + need.sum()) + spare
    order = rng.permutation(blocks).astype(np.int32)
    table = np.full((R, int((held + need).max()) + 1), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    ring = np.full(max(1, blocks), -1, np.int32)
    head = int(rng.integers(0, ring.size))
    free = order[at:]
    ring[(head + np.arange(free.size)) % ring.size] = free
    tokens = int(np.maximum(added, 0).sum()) + extra
    return lengths, added, table, ring, np.array([head, free.size], np.int32), tokens


def run_tables(lengths, added, table, ring, state, block, tokens, what):
    announce(f"kv_tables {what}: {lengths.size} requests, block {block}, {tokens} tokens")
    want = kv_ref.tables(lengths, added, table, ring, state, block, tokens)
    t, g = dev(table), dev(ring)
    out = nq.kv_tables(dev(lengths), dev(added), t, g, dev(state), block, tokens)
    torch.cuda.synchronize()
    got = (t, g, out.lengths, out.token_start, out.slots, out.free_state)
    for name, a, b in zip(("table", "ring", "lengths", "token_start", "slots", "free_state"), got, want):
        assert np.array_equal(a.cpu().numpy(), b), f"{what}: {name}"
    assert int(out.status) == want[6], what
    return want[6]


@pytest.mark.parametrize("R, longest, newest, ends, extra", [
    (1, 0, 0, 0, 0), (1, 0, 1, 0, 0), (1, 100, 1, 0, 3), (2, 70, 40, 1, 0), (48, 600, 1, 2, 9), (255, 90, 3, 7, 0),
    (256, 90, 3, 7, 1), (257, 90, 3, 7, 2), (1000, 300, 9, 60, 100), (3, 2000, 3001, 0, 0), (700, 40, 0, 700, 5)])
@pytest.mark.parametrize("block", [16, 128])
def test_tables(R, longest, newest, ends, extra, block):
    rng = np.random.default_rng(R * 7 + block)
    args = step(rng, R, longest, block, newest, ends, int(rng.integers(0, 9)), extra)
    assert run_tables(*args[:5], block, args[5], "step") == 0


def test_tables_refuse_on_the_gpu():
    """Each status bit; nothing is written."""
    rng = np.random.default_rng(5)
    lengths, added, table, ring, state, tokens = step(rng, 40, 200, 16, 60, 3, 2, 4)
    less = state - np.array([0, 3], np.int32)
    assert run_tables(lengths, added, table, ring, less, 16, tokens, "few blocks") == 1
    for r, bad in ((3, -1), (39, 2 ** 31 - 1), (0, table.shape[1] * 16 + 1)):
        x = lengths.copy()
        x[r] = bad
        st = run_tables(x, np.where(np.arange(40) == r, 1, added).astype(np.int32), table, ring, state, 16, tokens, "length")
        assert st & 2
    x = added.copy()
    x[7] = -2
    assert run_tables(lengths, x, table, ring, state, 16, tokens, "added") & 2
    assert run_tables(lengths, added, table, ring, state, 16, tokens - 5, "tokens") == 4
    for s in ([-1, 4], [ring.size, 4], [0, -1]):
        assert run_tables(lengths, added, table, ring, np.array(s, np.int32), 16, tokens, "ring") & 8
    short = ring[:40].copy()  # what comes back does not fit
    st = run_tables(np.full(40, 100, np.int32), np.full(40, -1, np.int32), table, short, np.array([0, 40], np.int32),
                    16, 0, "returns")
    assert st == 8


def test_tables_ring_shorter_than_the_pool():
    """Returned blocks that land on entries this step takes."""
    lengths = np.array([31, 160, 5, 64], np.int32)
    added = np.array([90, -1, 40, -1], np.int32)
    table = np.arange(4 * 12, dtype=np.int32).reshape(4, 12) + 100
    ring = np.arange(16, dtype=np.int32)
    state = np.array([5, 14], np.int32)
    assert run_tables(lengths, added, table, ring, state, 16, 1500, "short ring, too many back") == 8  # 14 - 8 + 14
    added[3] = 0
    assert run_tables(lengths, added, table, ring, state, 16, 1500, "short ring") == 0  # 14 - 8 + 10 = 16


def test_tables_strided_rows():
    rng = np.random.default_rng(8)
    lengths, added, table, ring, state, tokens = step(rng, 30, 200, 32, 40, 2, 3, 6)
    want = kv_ref.tables(lengths, added, table, ring, state, 32, tokens)
    wide = torch.full((30, table.shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    t = wide[:, 2:2 + table.shape[1]]
    t.copy_(dev(table))
    nq.kv_tables(dev(lengths), dev(added), t, dev(ring), dev(state), 32, tokens)
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert bool((wide[:, :2] == -7).all()) and bool((wide[:, -3:] == -7).all())


# --- store and load ---------------------------------------------------------------------------------------------

def slots_of(rng, past, new, block, spare=2):
    """Slots and starts of requests in shuffled blocks, and the number of blocks."""
    need = [-(-(p + n) // block) for p, n in zip(past, new)]
    order = rng.permutation(sum(need) + spare)
    slots, at = [], 0
    for p, n, b in zip(past, new, need):
        pos = np.arange(p, p + n)
        slots.append(order[at + pos // block] * block + pos % block)
        at += b
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return np.concatenate(slots).astype(np.int64), starts, order.size


def new_values(rng, n, heads, dim, dtype, wild=False):
    x = rng.normal(0, 1, (n, heads, dim)) * np.exp(rng.normal(0, 1, (n, heads, 1)))
    x[:, :, 5] *= 9
    if n > 2:
        x[1] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    if wild and n:
        t.view(-1)[:: 37] = float("nan")
        t.view(-1)[5:: 91] = float("inf")
        t.view(-1)[9:: 97] = -float("inf")
    return t


@pytest.mark.parametrize("code", ["q8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("block, dim, heads", [(16, 64, 3), (32, 128, 2), (64, 128, 1), (64, 256, 2), (128, 64, 2), (128, 256, 1)])
def test_store_and_load(code, dtype, block, dim, heads):
    """Prompts, single tokens and whole blocks into an arbitrary pool; every word of the pool afterwards."""
    rng = np.random.default_rng(block * dim + heads)
    past = [0, block - 1, 3, block, 2 * block + 5, 7, 0]
    new = [2 * block + 3, 1, 1, block, 2, 0, 5]
    slots, starts, blocks = slots_of(rng, past, new, block)
    kc, vc, ks, vs = pool(rng, blocks, heads, block, dim, code, junk=False)
    cache = upload(kc, vc, ks, vs, code)
    n = int(starts[-1])
    k, v = (new_values(rng, n, heads, dim, dtype, wild=i == 1 and dtype == "f32") for i in range(2))
    announce(f"kv_store {code} {dtype} block {block} dim {dim} heads {heads}")
    status = nq.kv_store(cache, k.to(DEV), v.to(DEV), dev(slots), dev(starts))
    torch.cuda.synchronize()
    fin = kv_ref.store(kc, ks, k.float().numpy(), slots, code, False)
    fin &= kv_ref.store(vc, vs, v.float().numpy(), slots, code, True)
    assert int(status) == (0 if fin else 1)
    assert np.array_equal(cache.k_scale.cpu().numpy(), ks) and np.array_equal(cache.v_scale.cpu().numpy(), vs)
    same_words(cache.k, kc, "k codes")
    same_words(cache.v, vc, "v codes")
    ids = np.r_[rng.permutation(blocks), 0, 0].astype(np.int32)
    for out in DT:
        gk, gv = nq.kv_load(cache, dev(ids), DT[out])
        torch.cuda.synchronize()
        for got, c, s, last in ((gk, kc, ks, False), (gv, vc, vs, True)):
            want = torch.from_numpy(kv_ref.load(c, s, ids, code, last)).to(DT[out])
            assert got.shape == want.shape and torch.equal(got.cpu(), want), (out, last)


@pytest.mark.parametrize("code", ["q8", "e4m3"])
def test_store_token_by_token(code):
    """A block that fills one token at a time, each step with its own scale, and from a strided projection."""
    rng = np.random.default_rng(3)
    heads, dim, block = 2, 64, 16
    kc, vc, ks, vs = pool(rng, 3, heads, block, dim, code, junk=False)
    cache = upload(kc, vc, ks, vs, code)
    fused = torch.from_numpy(rng.normal(0, 1, (20, 7 * dim + 1)).astype(np.float32)).to(DEV)
    for t in range(20):
        row = fused[t:t + 1]
        k = row[:, 1:1 + 2 * dim].view(1, heads, dim)  # an odd element offset: no vector loads
        v = row[:, 1 + 3 * dim:1 + 7 * dim].view(1, 2 * heads, dim)[:, ::2]
        k, v = k * float(1 + t % 5), v
        slots = np.array([(2 if t < 16 else 0) * block + t % 16], np.int64)
        nq.kv_store(cache, k, v, dev(slots), dev(np.array([0, 1], np.int32)))
        kv_ref.store(kc, ks, k.cpu().numpy(), slots, code, False)
        kv_ref.store(vc, vs, v.cpu().numpy(), slots, code, True)
    torch.cuda.synchronize()
    assert np.array_equal(cache.k_scale.cpu().numpy(), ks) and np.array_equal(cache.v_scale.cpu().numpy(), vs)
    same_words(cache.k, kc, "k")
    same_words(cache.v, vc, "v")


def test_store_refuses_bad_slots_on_the_gpu():
    """Slots outside the pool or out of order: status 2, the pool unchanged; the other requests are stored."""
    rng = np.random.default_rng(4)
    heads, dim, block = 2, 128, 32
    past, new = [0, 5, 9, 31, 40], [3, 4, 1, 2, 6]
    good, starts, blocks = slots_of(rng, past, new, block)
    for at, bad in ((0, -1), (0, -2 ** 63), (2, 7), (3, blocks * block), (3, 2 ** 62), (7, 2 ** 31), (9, 3), (12, 999)):
        kc, vc, ks, vs = pool(rng, blocks, heads, block, dim, "q8", junk=False)
        cache = upload(kc, vc, ks, vs, "q8")
        slots = good.copy()
        slots[at] = bad
        n = int(starts[-1])
        k, v = (new_values(rng, n, heads, dim, "bf16") for _ in range(2))
        announce(f"kv_store slot {at} = {bad}")
        status = nq.kv_store(cache, k.to(DEV), v.to(DEV), dev(slots), dev(starts))
        torch.cuda.synchronize()
        assert int(status) == 2
        r = int(np.searchsorted(starts, at, side="right")) - 1
        keep = np.ones(n, bool)
        keep[starts[r]:starts[r + 1]] = False
        kv_ref.store(kc, ks, k.float().numpy()[keep], good[keep], "q8", False)
        kv_ref.store(vc, vs, v.float().numpy()[keep], good[keep], "q8", True)
        mine = np.unique(good[~keep] // block)
        other = np.setdiff1d(np.arange(blocks), mine)
        got = cache.k.cpu().view(torch.uint8).numpy(), cache.v.cpu().view(torch.uint8).numpy()
        assert np.array_equal(got[0][other], kc[other]) and np.array_equal(got[1][other], vc[other])
        if mine.size == 1:
            assert np.array_equal(got[0][mine], kc[mine]) and np.array_equal(got[1][mine], vc[mine])


def test_load_ids_outside_the_pool():
    rng = np.random.default_rng(6)
    cache = upload(*pool(rng, 4, 2, 16, 64, "e4m3"), "e4m3")
    k, v = nq.kv_load(cache, dev(np.array([-1, 4, 2 ** 31 - 1, -2 ** 31], np.int32)), torch.float16)
    torch.cuda.synchronize()
    assert bool((k == 0).all()) and bool((v == 0).all())
    k, v = nq.kv_load(cache, dev(np.zeros(0, np.int32)))
    assert k.shape == (0, 16, 2, 64)


# --- attention --------------------------------------------------------------------------------------------------

def attention_case(rng, past, new, heads, group, dim, block, code, dtype, holes=0, pad=0, spread=1.0):
    """A pool of arbitrary words in which just the requests' keys are sound, their tables and queries."""
    total = [p + n for p, n in zip(past, new)]
    need = [-(-max(t, 0) // block) for t in total]
    blocks = sum(need) + 3
    order = rng.permutation(blocks)
    kc, vc, ks, vs = pool(rng, blocks, heads, block, dim, code)
    good = pool(rng, blocks, heads, block, dim, code, junk=False)
    table = np.full((len(past), max(need + [1]) + 1), -1, np.int32)
    used = np.zeros(blocks, bool)
    at = 0
    for r, (t, b) in enumerate(zip(total, need)):
        table[r, :b] = order[at:at + b]
        for j in range(b):
            live = min(block, t - j * block)
            i = order[at + j]
            kc[i, :, :live], vc[i, :, :, :live] = good[0][i, :, :live], good[1][i, :, :, :live]
            used[i] = True
        table[r, b:] = rng.choice([-1, 0, blocks, 2 ** 31 - 1, -2 ** 31], table.shape[1] - b)
        if holes and b > 2:
            table[r, rng.integers(0, b, holes)] = rng.choice([-1, blocks + 5], holes)
        at += b
    ks[~used], vs[~used] = np.nan, np.inf
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(starts[-1]) + pad
    q = rng.normal(0, spread, (n, heads * group, dim)).astype(np.float32)
    q = torch.from_numpy(q).to(DT[dtype])
    return (kc, vc, ks, vs), q, starts, np.array(total, np.int32), table


def run_attention(case, code, dtype, window, what, scale=None, max_new=None, max_length=None):
    host, q, starts, lengths, table = case
    kc, vc, ks, vs = host
    dim = kc.shape[3]
    scale = dim ** -0.5 if scale is None else scale
    announce(f"kv_attention {what}")
    cache = upload(*host, code)
    out, lse = nq.kv_attention(cache, q.to(DEV), dev(starts), dev(lengths), dev(table), scale=scale, window=window,
                               max_new=max_new, max_length=max_length, return_lse=True)
    torch.cuda.synchronize()
    assert out.dtype == q.dtype and out.shape == q.shape
    ref = kv_ref.attention(host, code, q.float().numpy(), starts, lengths, table, float(np.float32(scale)), window)
    worst = kv_ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, dtype,
                                   int(max(lengths)) if len(lengths) else 0, dim, what)
    announce(f"  {worst:.3f} of the bound")
    return out, lse


@pytest.mark.parametrize("code", ["q8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_attention_decode(code, dtype, dim, block):
    """One new token, lengths from one up to several tiles."""
    rng = np.random.default_rng(dim + block)
    past = [0, 1, 14, 15, 16, 62, 63, 64, 65, 255, 256, 300, 511, 700]
    case = attention_case(rng, past, [1] * len(past), 2, 4, dim, block, code, dtype)
    run_attention(case, code, dtype, 0, f"decode {code} {dtype} dim {dim} block {block}", max_new=1)


@pytest.mark.parametrize("code, dtype, heads, group, dim, block", [
    ("q8", "bf16", 1, 1, 64, 16), ("q8", "f16", 3, 5, 128, 32), ("e4m3", "bf16", 2, 16, 128, 64),
    ("e4m3", "f32", 2, 3, 64, 128), ("q8", "f32", 1, 8, 256, 16), ("e4m3", "f16", 1, 2, 256, 64),
    ("q8", "bf16", 4, 40, 64, 32)])
@pytest.mark.parametrize("window", [0, 1, 37, 200])
def test_attention_mixed(code, dtype, heads, group, dim, block, window):
    """Prompts, drafted tokens, single tokens, requests without new tokens; windows; tokens of no request."""
    rng = np.random.default_rng(heads * 100 + group + window)
    past = [0, 0, 130, 3, 77, 500, 0, 64, 250]
    new = [1, 97, 5, 0, 17, 1, 33, 64, 3]
    case = attention_case(rng, past, new, heads, group, dim, block, code, dtype, pad=3)
    run_attention(case, code, dtype, window, f"mixed {code} {dtype} group {group} dim {dim} block {block} w {window}")


@pytest.mark.parametrize("code", ["q8", "e4m3"])
@pytest.mark.parametrize("window", [0, 700])
def test_attention_pieces(code, window):
    """Long rows in several pieces, with table entries that name no block."""
    rng = np.random.default_rng(11)
    case = attention_case(rng, [3000, 511, 1025, 40], [1, 2, 1, 4], 2, 4, 128, 64, code, "bf16", holes=3)
    run_attention(case, code, "bf16", window, f"pieces {code} w {window}", max_new=4)
    case = attention_case(rng, [2047, 4500], [1, 1], 1, 8, 64, 16, code, "f32", holes=9)
    run_attention(case, code, "f32", window, f"pieces f32 {code} w {window}", max_new=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_prompt_in_pieces(dtype):
    """Many rows over many keys with one head."""
    rng = np.random.default_rng(12)
    case = attention_case(rng, [900], [150], 1, 2, 128, 32, "q8", dtype)
    run_attention(case, "q8", dtype, 0, f"prompt {dtype}", max_new=150, max_length=1050)


@pytest.mark.parametrize("requests", [2, 17, 256, 300])
def test_attention_many_requests(requests):
    """Chunks and single tokens of many requests in one call (the longest of up to 256 start first)."""
    rng = np.random.default_rng(requests)
    new = [int(rng.choice([1, 1, 1, 3, 140 if r % 16 == 1 else 2])) for r in range(requests)]
    new[1] = 150
    past = [int(rng.integers(0, 90)) for _ in new]
    past[0] = past[-1] = 70
    case = attention_case(rng, past, new, 1, 1, 64, 16, "q8", "bf16")
    run_attention(case, "q8", "bf16", 0, f"{requests} requests", max_new=max(new))


@pytest.mark.parametrize("code, dim, block", [("q8", 64, 64), ("q8", 128, 16), ("e4m3", 256, 32)])
def test_attention_chunks_in_a_graph(code, dim, block):
    """Chunks of changing lengths under one captured call, against the eager calls, bit for bit."""
    rng = np.random.default_rng(dim)
    host, q, starts, lengths, table = attention_case(rng, [300, 20, 150], [80, 90, 5], 2, 4, dim, block, code, "f16")
    cache = upload(*host, code)
    qd, s, n, t = q.to(DEV), dev(starts), dev(lengths), dev(table)
    call = lambda: nq.kv_attention(cache, qd, s, n, t, max_new=90, max_length=400, return_lse=True)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for trial in range(4):
        n.copy_(dev(lengths - np.array([31, 0, 7], np.int32) * trial))
        s.copy_(dev(np.array([0, 80 - 20 * trial, 170 - 20 * trial, 175 - 20 * trial], np.int32)))
        eager = call()
        held[0].fill_(7), held[1].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], eager[0]) and torch.equal(held[1], eager[1]), trial
        torch.randn(1000, device=DEV).sum().item()


def test_attention_rows_without_keys():
    """More new tokens than the length, a length of 0, tables without blocks."""
    rng = np.random.default_rng(13)
    host, q, starts, lengths, table = attention_case(rng, [0, 20, 50], [30, 4, 2], 2, 2, 64, 16, "q8", "bf16")
    lengths = np.array([7, 0, 52], np.int32)
    table[2] = -1
    out, lse = run_attention((host, q, starts, lengths, table), "q8", "bf16", 0, "empty rows")
    assert int(torch.isneginf(lse).sum()) == (23 + 4 + 2) * 4


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_attention_sharp_and_uneven(dtype):
    """Large scores, queries of very different size, one dominant key, scales that differ by 2^40 between blocks."""
    rng = np.random.default_rng(14)
    host, q, starts, lengths, table = attention_case(rng, [400, 90], [3, 40], 2, 4, 128, 16, "q8", dtype)
    host[3][table[0, 3]] *= np.float32(2.0 ** 20)
    host[3][table[0, 9]] *= np.float32(2.0 ** -20)
    q = (q.float() * torch.logspace(-3, 1, q.shape[0])[:, None, None]).to(q.dtype)
    q[0, 0] = 0
    run_attention((host, q, starts, lengths, table), "q8", dtype, 0, f"sharp {dtype}")


def test_attention_strided_queries_and_table():
    rng = np.random.default_rng(15)
    host, q, starts, lengths, table = attention_case(rng, [100, 7, 64], [1, 9, 2], 2, 4, 128, 32, "e4m3", "bf16")
    cache = upload(*host, "e4m3")
    a = (dev(starts), dev(lengths))
    want = nq.kv_attention(cache, q.to(DEV), *a, dev(table))
    wide = torch.zeros((q.shape[0], 3 * 8 * 128 + 1), dtype=q.dtype, device=DEV)
    view = wide[:, 1:1 + 2 * 8 * 128].view(q.shape[0], 16, 128)[:, ::2]
    view.copy_(q)
    t = torch.full((3, table.shape[1] + 4), 1, dtype=torch.int32, device=DEV)
    t[:, 1:1 + table.shape[1]] = dev(table)
    got = nq.kv_attention(cache, view, *a, t[:, 1:1 + table.shape[1]])
    assert torch.equal(got, want)


def test_attention_is_deterministic_on_other_streams_and_in_graphs():
    rng = np.random.default_rng(16)
    host, q, starts, lengths, table = attention_case(rng, [1500, 600, 30], [1, 1, 1], 2, 4, 128, 64, "q8", "bf16")
    cache = upload(*host, "q8")
    qd, s, n, t = q.to(DEV), dev(starts), dev(lengths), dev(table)
    call = lambda **kw: nq.kv_attention(cache, qd, s, n, t, max_new=1, return_lse=True, **kw)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [call(stream=side) for _ in range(3)]
    side.synchronize()
    for o, e in got:
        assert torch.equal(o, want[0]) and torch.equal(e, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for trial in range(4):
        shorter = dev(np.array([1501 - 300 * trial, 601, 31 - trial], np.int32))
        n.copy_(shorter)
        eager = call()
        held[0].fill_(7), held[1].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], eager[0]) and torch.equal(held[1], eager[1]), trial


def test_step_in_a_graph():
    """Tables, store and attention of a step captured together, replayed against the eager calls."""
    rng = np.random.default_rng(17)
    heads, dim, block = 2, 64, 16
    k, v = (torch.randn((5, heads, dim), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((5, 4 * heads, dim), device=DEV, dtype=torch.bfloat16)
    host = pool(rng, 12, heads, block, dim, "q8", junk=False)

    def fresh():
        table = dev(np.array([[3, 4, -1, -1], [5, -1, -1, -1], [6, -1, -1, -1]], np.int32))
        ring = dev(np.array([7, 8, 9, 10] + [0] * 8, np.int32))
        return upload(*[x.copy() for x in host], "q8"), table, ring

    def one(cache, table, ring):
        st = nq.kv_tables(lengths, added, table, ring, state, block, 5)
        bad = nq.kv_store(cache, k, v, st.slots, st.token_start)
        return st, bad, nq.kv_attention(cache, q, st.token_start, st.lengths, table, max_new=4)

    lengths, added = dev(np.array([32, 3, 9], np.int32)), dev(np.array([1, 3, -1], np.int32))
    state = dev(np.array([0, 4], np.int32))
    st, bad, want = one(*fresh())
    torch.cuda.synchronize()
    assert int(st.status) == 0 and int(bad) == 0
    cache, table, ring = fresh()
    start = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, table, ring)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gst, gbad, got = one(cache, table, ring)
    for _ in range(4):
        for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, table, ring), start):
            x.copy_(y)
        got.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and int(gst.status) == 0 and int(gbad) == 0
        assert torch.equal(gst.slots, st.slots) and torch.equal(gst.lengths, st.lengths)
        torch.randn(1000, device=DEV).sum().item()


@pytest.mark.parametrize("code", ["q8", "e4m3"])
def test_example_serving_loop(code):
    """examples/kv_serving.py: no status bit, and the last step is attention over what the cache holds (both sides
    round to bfloat16's or binary32's precision: within two bfloat16 steps of the largest output)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv_serving.py")
    spec = importlib.util.spec_from_file_location("kv_serving", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    announce(f"serving loop {code}")
    problems, worst = example.main(requests=5, steps=12, code=code, prompt=150)
    assert problems == 0 and worst < 2 * torch.finfo(torch.bfloat16).eps


def test_attention_pool_past_32_bits():
    """Blocks whose code offsets pass 2^32 bytes."""
    heads, dim, block = 8, 128, 128
    blocks = 2 ** 32 // (heads * dim * block) + 40
    cache = nq.KvCache.empty(blocks, heads, block, dim, "q8", DEV)
    rng = np.random.default_rng(18)
    ids = np.array([blocks - 1, 3, blocks - 20, blocks - 2, 2 ** 31 // (heads * dim * block) + 1], np.int32)
    past, n = 4 * block + 17, 40
    slots = (ids[np.arange(past + n) // block].astype(np.int64) * block + np.arange(past + n) % block)
    x = [new_values(rng, past + n, heads, dim, "bf16") for _ in range(2)]
    announce(f"kv pool of {blocks} blocks")
    nq.kv_store(cache, x[0].to(DEV), x[1].to(DEV), dev(slots), dev(np.array([0, past + n], np.int32)))
    small = upload(*pool(rng, 5, heads, block, dim, "q8", junk=False), "q8")
    near = (np.arange(5)[np.arange(past + n) // block] * block + np.arange(past + n) % block).astype(np.int64)
    nq.kv_store(small, x[0].to(DEV), x[1].to(DEV), dev(near), dev(np.array([0, past + n], np.int32)))
    far_k, far_v = nq.kv_load(cache, dev(ids[:4]))
    near_k, near_v = nq.kv_load(small, dev(np.arange(4, dtype=np.int32)))
    assert torch.equal(far_k, near_k) and torch.equal(far_v, near_v)
    q = torch.randn((n, 16, dim), device=DEV, dtype=torch.bfloat16)
    a = (dev(np.array([0, n], np.int32)), dev(np.array([past + n], np.int32)))
    far = nq.kv_attention(cache, q, *a, dev(ids[None]))
    assert torch.equal(far, nq.kv_attention(small, q, *a, dev(np.arange(5, dtype=np.int32)[None])))


def test_binding_refuses():
    rng = np.random.default_rng(19)
    cache = upload(*pool(rng, 3, 2, 16, 64, "q8"), "q8")
    i32 = lambda *x: dev(np.array(x, np.int32))  # noqa: E731
    q = torch.zeros((2, 4, 64), device=DEV, dtype=torch.bfloat16)
    table = dev(np.zeros((1, 2), np.int32))
    for bad in (q[..., :32], q[0], q.cpu(), q.transpose(1, 2)):
        with pytest.raises(ValueError, match="q must"):
            nq.kv_attention(cache, bad, i32(0, 2), i32(2), table)
    with pytest.raises(ValueError, match="token_start"):
        nq.kv_attention(cache, q, i32(0, 1, 2), i32(2), table)
    with pytest.raises(ValueError, match="table"):
        nq.kv_attention(cache, q, i32(0, 2), i32(2), table.long())
    with pytest.raises(ValueError, match="lengths"):
        nq.kv_attention(cache, q, i32(0, 2), i32(2).long(), table)
    with pytest.raises(nq.NqError, match="BAD_DIM"):
        nq.kv_attention(cache, q[:, :3], i32(0, 2), i32(2), table)
    with pytest.raises(nq.NqError, match="BAD_DTYPE"):
        nq.kv_attention(cache, q.double(), i32(0, 2), i32(2), table)
    with pytest.raises(ValueError, match="k must"):
        nq.kv_store(cache, q, q, dev(np.zeros(2, np.int64)), i32(0, 2))
    with pytest.raises(ValueError, match="slots"):
        nq.kv_store(cache, q[:, :2], q[:, :2], i32(0, 1), i32(0, 2))
    with pytest.raises(ValueError, match="one type"):
        nq.kv_store(cache, q[:, :2], q[:, :2].float(), dev(np.zeros(2, np.int64)), i32(0, 2))
    with pytest.raises(ValueError, match="ids"):
        nq.kv_load(cache, dev(np.zeros(2, np.int64)))
