"""GPU: the 8-bit key/value cache where its inputs or bounds reach the ends of their ranges, against plain
implementations."""
import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import kv_ref
from gpu_util import announce
from kv_ref import DT
from test_gpu_kv import DEV, attention_case, dev, upload

pytestmark = pytest.mark.gpu
TINY = np.float32(2.0 ** -126)  # the scale that the store gives a block of zeros


def attend(case, code, dtype, what, window=0, max_new=None, max_length=None, scale=None, ref=None, keys=None):
    """A call against the reference (kv_ref.attention unless given), within kv_ref.check_attention's bound."""
    host, q, starts, lengths, table = case
    dim = host[0].shape[3]
    scale = dim ** -0.5 if scale is None else scale
    announce(f"kv_attention {what}")
    cache = upload(*host, code)
    out, lse = nq.kv_attention(cache, q.to(DEV), dev(starts), dev(lengths), dev(table), scale=scale, window=window,
                               max_new=max_new, max_length=max_length, return_lse=True)
    torch.cuda.synchronize()
    if ref is None:
        ref = kv_ref.attention(host, code, q.float().numpy(), starts, lengths, table, float(np.float32(scale)), window,
                               max_length)
        if max_new is not None:  # rows past it: no output
            at = np.concatenate([np.arange(s0 + max_new, s1) for s0, s1 in zip(starts, starts[1:])] + [[]]).astype(int)
            ref[0][at], ref[1][at], ref[2][at] = 0, -np.inf, 0
    kv_ref.check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, dtype,
                           int(max(lengths)) if keys is None else keys, dim, what)


# dim and heads that leave the rows' keys in one piece or cut them in two of about 20000
@pytest.mark.parametrize("dim, heads", [(64, 128), (64, 64), (128, 128), (128, 64), (256, 64), (256, 32)])
@pytest.mark.parametrize("tail", [0, 300])
@pytest.mark.parametrize("code, dtype", [("q8", "bf16"), ("e4m3", "f16")])
def test_zero_heads_over_long_contexts(dim, heads, tail, code, dtype):
    """Keys of zero, and values of zero up to the last `tail` keys: every weight is equal, so a row's output is the
    mean of its values and lse = ln(keys)."""
    rng = np.random.default_rng(dim + heads + tail)
    block, new, length, past_zero = 64, 150, [40000, 39937], 39000 if tail else 40000
    blocks = 1 + -(-(40000 - past_zero) // block)
    kc = np.zeros((blocks, heads, block, dim), np.uint8)
    vc = np.zeros((blocks, heads, dim, block), np.uint8)
    ks, vs = (np.full((blocks, heads), TINY) for _ in range(2))
    vc[1:] = rng.integers(0, 100, vc[1:].shape)
    vs[1:] = rng.uniform(0.01, 0.03, vs[1:].shape).astype(np.float32)
    first = past_zero // block  # the table entry of the first value that may not be 0
    row = np.zeros(-(-40000 // block), np.int32)
    row[first:] = 1 + np.arange(row.size - first)
    starts = np.array([0, new, 2 * new], np.int32)
    q = torch.from_numpy(rng.normal(0, 1, (2 * new, heads, dim)).astype(np.float32)).to(DT[dtype])
    v = kv_ref.code_values(vc[1:], code) * vs[1:].astype(np.float64)[:, :, None, None]
    sums = np.concatenate([np.zeros((1, heads, dim)), v.transpose(0, 3, 1, 2).reshape(-1, heads, dim).cumsum(0)])
    seen = np.concatenate([np.arange(n - new, n) + 1 for n in length])
    out = sums[np.maximum(seen - first * block, 0)] / seen[:, None, None]
    lse = np.broadcast_to(np.log(seen)[:, None], (2 * new, heads))
    case = (kc, vc, ks, vs), q, starts, np.array(length, np.int32), np.stack([row, row])
    attend(case, code, dtype, f"zero heads dim {dim} heads {heads} tail {tail} {code}", max_new=new,
           ref=(out, lse, out, np.zeros((2 * new, heads))))


@pytest.mark.parametrize("code, dtype", [("q8", "bf16"), ("e4m3", "f16"), ("q8", "f32")])
@pytest.mark.parametrize("dim, block", [(64, 64), (128, 16), (256, 32)])
@pytest.mark.parametrize("window", [0, 45])
def test_zero_keys_at_the_edge(code, dtype, dim, block, window):
    """Blocks of zero keys (scale 2^-126) where the mask ends, values as usual, small queries: the factor of their
    scores is below binary32's range."""
    rng = np.random.default_rng(dim + window)
    host, q, starts, lengths, table = attention_case(rng, [90, 7, 0], [150, 133, 1], 2, 2, dim, block, code, dtype,
                                                     spread=1e-3)
    for r, n in enumerate(lengths):
        for j in range(0 if r == 1 else n // block // 2, -(-n // block)):  # the second half, or all
            host[0][table[r, j]], host[2][table[r, j]] = 0, TINY
    attend((host, q, starts, lengths, table), code, dtype, f"zero keys {code} {dtype} dim {dim} w {window}", window,
           max_new=150)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new", [3, 150])
def test_large_factor_of_zero_scores(dtype, new):
    """A channel in which the queries are huge and every key is zero: scores of 0 times a factor above binary32's
    range."""
    rng = np.random.default_rng(new)
    host, q, starts, lengths, table = attention_case(rng, [100], [new], 2, 1, 64, 16, "q8", dtype)
    host[0][:, :, :, 5] = 0
    host[2][:] = 1e9
    q[:] = 0
    q[:, :, 5] = 3e38
    attend((host, q, starts, lengths, table), "q8", dtype, f"large factor {dtype} {new}", max_new=new)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("max_new, max_length", [(1, None), (40, None), (200, 150), (200, 1), (140, 333), (60, 171)])
def test_bounds_below_the_requests(dtype, group, window, max_new, max_length):
    """max_new and max_length below a request's new tokens and length: the rows within max_new keep their positions,
    those past it are 0 with a sum of 0, keys from max_length on are not seen."""
    rng = np.random.default_rng(max_new + window)
    case = attention_case(rng, [100, 0, 33, 0], [150, 151, 5, 64], 2, group, 64, 32, "q8", dtype, pad=2)
    attend(case, "q8", dtype, f"bounds {max_new} {max_length} {dtype} group {group} w {window}", window, max_new,
           max_length)


@pytest.mark.parametrize("count, need", [(15, 12), (15, 5), (11, 1), (2 ** 31 - 1, 11)])
def test_tables_refuse_a_count_above_the_ring(count, need):
    """More free blocks than a ring of 10 holds cannot be: status 8 and nothing changes, whatever the step takes."""
    ring = np.arange(10, dtype=np.int32)
    table = np.full((2, 12), -1, np.int32)
    added = np.array([need * 16 - 32, 20], np.int32) if need > 2 else np.array([0, 16], np.int32)
    announce(f"kv_tables count {count} need {need}")
    t, g = dev(table), dev(ring)
    step = nq.kv_tables(dev(np.zeros(2, np.int32)), dev(added), t, g, dev(np.array([3, count], np.int32)), 16, 200)
    torch.cuda.synchronize()
    assert int(step.status) == 8
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(g.cpu().numpy(), ring)
    assert step.lengths.tolist() == [0, 0] and step.token_start.tolist() == [0, 0, 0]
    assert step.free_state.tolist() == [3, count] and bool((step.slots == -1).all())


@pytest.mark.parametrize("code, dtype, dim", [("q8", "bf16", 64), ("e4m3", "f16", 128)])
@pytest.mark.parametrize("window", [0, 1500])
def test_pieces_beside_a_chunk(code, dtype, dim, window):
    """Few rows over several pieces in a call whose chunk has more tokens than the few-rows kernel takes: the pieces
    have a place for each request's few tokens, not for each token of the call."""
    rng = np.random.default_rng(dim + window)
    case = attention_case(rng, [2300, 1900, 20, 3100], [1, 60, 16, 2], 1, 8, dim, 32, code, dtype, holes=2)
    attend(case, code, dtype, f"pieces beside a chunk {code} {dtype} w {window}", window, max_new=60)


@pytest.mark.parametrize("requests, filled", [(257, 257), (1000, 1000), (70000, 70000), (1 << 20, 3000)])
def test_store_of_many_requests(requests, filled):
    """One call for all requests stores what calls of 200 requests store."""
    rng = np.random.default_rng(requests)
    heads, dim, block = 1, 64, 16
    new = np.zeros(requests, np.int64)
    new[rng.permutation(requests)[:filled]] = rng.choice([0, 1, 1, 1, 2, 17], filled)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(starts[-1])
    at = rng.permutation(2 * filled)  # two blocks for each request that may have tokens
    first = np.zeros(requests, np.int64)
    first[np.nonzero(new)[0]] = np.arange(np.count_nonzero(new))
    off = rng.integers(0, block, requests)
    r = np.repeat(np.arange(requests), new)
    pos = off[r] + np.arange(n) - starts[r]  # 15 + 17 tokens at most
    slots = at[2 * first[r] + pos // block] * block + pos % block
    k, v = (torch.randn((n, heads, dim), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    caches = []
    for _ in range(2):
        c = nq.KvCache.empty(2 * filled, heads, block, dim, "q8", DEV)
        for x in (c.k, c.v, c.k_scale, c.v_scale):
            x.fill_(1)
        caches.append(c)
    announce(f"kv_store of {requests} requests, {n} tokens")
    s, t = dev(slots.astype(np.int64)), dev(starts)
    status = nq.kv_store(caches[0], k, v, s, t)
    torch.cuda.synchronize()
    assert int(status) == 0
    used = np.nonzero(new)[0]
    for i in range(0, used.size, 200):
        part = used[i:i + 200]
        a, b = int(starts[part[0]]), int(starts[part[-1] + 1])
        own = np.concatenate([[0], np.cumsum(new[part])]).astype(np.int32)
        nq.kv_store(caches[1], k[a:b], v[a:b], s[a:b], dev(own))
    torch.cuda.synchronize()
    for x, y in zip((caches[0].k, caches[0].v, caches[0].k_scale, caches[0].v_scale),
                    (caches[1].k, caches[1].v, caches[1].k_scale, caches[1].v_scale)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("code", ["q8", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_values_near_the_least_scale(code, new):
    """Value scales of 2^-112 and a channel in which the first 64 keys, whose weights are e^12 times the others', are 0:
    binary32 outputs of about 2^-122 there, in full precision."""
    rng = np.random.default_rng(new)
    host, q, starts, lengths, table = attention_case(rng, [330, 280], [new, new], 2, 4, 64, 32, code, "f32")
    kc, vc, ks, vs = host
    q[:] = 1
    for row in table:
        for j, b in enumerate(row[: -(-330 // 32)]):
            if 0 <= b < ks.shape[0]:
                kc[b] = (1 if code == "q8" else 0x38) if j < 2 else 0
                ks[b] = 1.5
                if j < 2:
                    vc[b, :, :8] = 0
    vs[np.isfinite(vs)] = 2.0 ** -112
    attend((host, q, starts, lengths, table), code, "f32", f"least scales {code} {new}", max_new=new)
