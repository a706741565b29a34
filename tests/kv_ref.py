"""Plain implementations of the 8-bit key/value cache operators (numpy; binary32 where the definition names it, else
binary64), and builders of small caches."""
import numpy as np
import torch

QMAX = {"q8": np.float32(127), "e4m3": np.float32(448)}
TINY = np.float32(2.0 ** -126)
CODE_DT = {"q8": torch.int8, "e4m3": torch.float8_e4m3fn}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def e4m3_values():
    """The 256 E4M3FN values (NaN for 0x7F and 0xFF), from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


E4M3 = e4m3_values()


def code_values(codes, code):
    """uint8 words as the numbers they stand for (float64)."""
    return codes.view(np.int8).astype(np.float64) if code == "q8" else E4M3[codes]


def to_codes(x, code):
    """binary32 values to uint8 words: nearest, ties to even, saturated."""
    x = x.astype(np.float64)
    if code == "q8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x), 448.0)
    grid = E4M3[:127]
    i = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    w = np.where(up, i, i - 1).astype(np.uint8)
    return np.where(np.signbit(x), w | 128, w).astype(np.uint8)


def tables(lengths, added, table, ring, state, block, tokens):
    """The step's tables, request by request."""
    table, ring = table.copy(), ring.copy()
    R, width = table.shape
    head, count = int(state[0]), int(state[1])
    held = [-(-int(x) // block) for x in lengths]
    need = [-(-(int(x) + max(int(a), 0)) // block) - h for x, a, h in zip(lengths, added, held)]
    give = [h if a < 0 else 0 for a, h in zip(added, held)]
    total = sum(max(int(a), 0) for a in added)
    status = 1 if sum(need) > count else 0
    if any(x < 0 or a < -1 or int(x) + max(int(a), 0) > width * block for x, a in zip(lengths, added)):
        status |= 2
    if total > tokens:
        status |= 4
    if count < 0 or head < 0 or head >= ring.size or count - sum(need) + sum(give) > ring.size:
        status |= 8
    slots = np.full(tokens, -1, np.int64)
    if status:
        return table, ring, lengths.copy(), np.zeros(R + 1, np.int32), slots, np.array(state), status
    starts, at, out = [0], head, lengths.copy()
    for r in range(R):
        for j in range(need[r]):
            table[r, held[r] + j] = ring[at % ring.size]
            at += 1
        n = max(int(added[r]), 0)
        for i in range(n):
            p = int(lengths[r]) + i
            slots[starts[-1] + i] = int(table[r, p // block]) * block + p % block
        starts.append(starts[-1] + n)
        out[r] = 0 if added[r] < 0 else lengths[r] + n
    tail = head + count
    for r in range(R):
        for j in range(give[r]):
            ring[tail % ring.size] = table[r, j]
            tail += 1
    state = np.array([(head + sum(need)) % ring.size, count - sum(need) + sum(give)], np.int32)
    return table, ring, out, np.array(starts, np.int32), slots, state, 0


def store(codes, scales, x, slots, code, tokens_last):
    """x [n, heads, dim] (float32) into codes (uint8 [blocks, heads, block, dim], or [.., dim, block] with
    tokens_last) and scales, in place; all arithmetic in binary32.  Returns whether every value was finite."""
    view = codes.swapaxes(2, 3) if tokens_last else codes
    block = view.shape[2]
    one = np.float32(1)
    x = x.astype(np.float32)
    finite = np.isfinite(x)
    for b in np.unique(slots // block):
        rows = np.nonzero(slots // block == b)[0]
        off = slots[rows] % block
        first = off.min()
        for h in range(x.shape[1]):
            vals = x[rows, h]
            amax = np.where(finite[rows, h], np.abs(vals), 0).max().astype(np.float32)
            old = scales[b, h] if first > 0 else np.float32(0)
            new = max(old, np.float32(amax / QMAX[code]), TINY)
            if first > 0 and new > old:
                was = code_values(view[b, h, :first], code).astype(np.float32)
                view[b, h, :first] = to_codes(was * np.float32(old / new), code)
            with np.errstate(over="ignore", invalid="ignore"):
                y = np.where(np.isnan(vals), 0, vals).astype(np.float32) * np.float32(one / new)
            view[b, h, off] = to_codes(np.clip(y, -1e30, 1e30), code)
            scales[b, h] = new
    return bool(finite.all())


def load(codes, scales, ids, code, tokens_last):
    """binary32 values [n, block, heads, dim]."""
    x = code_values(codes[ids], code).astype(np.float32) * scales[ids][:, :, None, None]
    return np.ascontiguousarray(x.transpose(0, 3, 1, 2) if tokens_last else x.swapaxes(1, 2))


def attention(cache, code, q, starts, lengths, table, scale, window, max_length=None):
    """Returns out, lse in binary64 and, for the error bound, the attended magnitude sum_j p_j |v_j| / sum_j p_j and
    the largest of scale |q| |k_j| over the row's keys.  cache: k, v (uint8), ks, vs."""
    kc, vc, ks, vs = cache
    blocks, heads, block, dim = kc.shape
    n, q_heads, _ = q.shape
    group = q_heads // heads
    out, lse = np.zeros((n, q_heads, dim)), np.full((n, q_heads), -np.inf)
    mag, size = np.zeros((n, q_heads, dim)), np.zeros((n, q_heads))
    for r, length in enumerate(lengths):
        s0, s1 = int(starts[r]), int(starts[r + 1])
        length = int(length)
        live = min(length, table.shape[1] * block, max_length or length)
        if s0 == s1 or live <= 0:
            continue
        ids = table[r, : -(-live // block)]
        named = (ids >= 0) & (ids < blocks)
        safe = np.where(named, ids, 0)
        known = np.repeat(named, block)[:live]
        for h in range(heads):
            k = (code_values(kc[safe, h], code) * ks[safe, h].astype(np.float64)[:, None, None]).reshape(-1, dim)[:live]
            v = (code_values(vc[safe, h], code) * vs[safe, h].astype(np.float64)[:, None, None])
            v = v.swapaxes(1, 2).reshape(-1, dim)[:live]
            for t in range(s1 - s0):
                pos = length - (s1 - s0) + t
                key = np.arange(live)
                see = known & (key <= pos)
                if window:
                    see &= key > pos - window
                if not see.any():
                    continue
                for g in range(group):
                    x = q[s0 + t, h * group + g].astype(np.float64)
                    s = scale * (k[see] @ x)
                    top = s.max()
                    p = np.exp(s - top)
                    i = (s0 + t, h * group + g)
                    out[i] = p @ v[see] / p.sum()
                    mag[i] = p @ np.abs(v[see]) / p.sum()
                    lse[i] = top + np.log(p.sum())
                    size[i] = abs(scale) * (np.abs(k[see]) @ np.abs(x)).max()
    return out, lse, mag, size


def check_attention(got_out, got_lse, ref, dtype, keys, dim, what):
    """The kernel's error bound.  Roundings of 2^-24 each: a score of dim products takes dim additions and at most
    8 more (the query's terms, the scales, the exponent's argument) of its magnitude `size`; a probability then
    has that relative error, twice (numerator and sum), 2 units of the exponential, one rounding to 2^-11 (2^-22 in
    two terms) and the sum over the keys one unit each with 16 for the joins.  The output is rounded once."""
    out, lse, mag, size = ref
    u = 2.0 ** -24
    term = 2.0 ** -22 if dtype == "f32" else 2.0 ** -11
    rel = 2 * np.expm1((dim + 8) * u * size) + term + (keys + 20) * u
    half = torch.finfo(DT[dtype]).eps / 2
    tol = rel[:, :, None] * mag * (1 + half) + half * np.abs(out) + 2.0 ** -24 * (dtype == "f16") + 1e-40
    err = np.abs(got_out - out)
    worst = np.max(err / tol) if err.size else 0.0
    assert np.isfinite(got_out).all() and (err <= tol).all(), f"{what}: out error {worst:.3g} of the bound"
    dead = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), dead), f"{what}: rows without keys"
    assert (got_out[dead] == 0).all(), f"{what}: rows without keys are not 0"
    tol = np.expm1((dim + 8) * u * size) + (keys + 20) * u + 4 * u * np.abs(np.where(dead, 0, lse))
    err = np.abs(np.where(dead, 0, got_lse) - np.where(dead, 0, lse))
    assert (err <= tol).all(), f"{what}: lse error {np.max(err / tol):.3g} of the bound"
    return float(worst)
