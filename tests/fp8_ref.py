"""Plain implementations of the E4M3 block operators and of the experts' rows (numpy; binary32 where the definition names
it, else binary64), and the error bounds that their kernels are held to."""
import numpy as np
import torch

from kv_ref import E4M3, to_codes

B = 128
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
LEAST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least subnormal


def quantize(x, tile=1):
    """Code words uint8 and scales of a binary32 [rows, cols] array."""
    rows, cols = x.shape
    bands = -(-rows // tile)
    wide = np.zeros((bands * tile, cols), np.float32)
    wide[:rows] = x
    wide = wide.reshape(bands, tile, cols // B, B)
    finite = np.isfinite(wide)
    amax = np.where(finite, np.abs(wide), 0).max((1, 3)).astype(np.float32)
    scales = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126)).astype(np.float32)
    inv = (np.float32(1) / scales).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.where(finite, wide, 0) * inv[:, None, :, None]
    words = np.where(finite, to_codes(y.astype(np.float32), "e4m3"), 0x7F).astype(np.uint8)
    return words.reshape(-1, cols)[:rows], scales


def numbers(words, scales, tile=1):
    """The numbers that codes and scales stand for, binary64 (exact products)."""
    wide = np.repeat(np.repeat(scales.astype(np.float64), tile, 0)[: words.shape[0]], B, 1)
    return E4M3[words] * wide


def product(xw, xs, ww, ws, wide_sums, waves=16):
    """y = x w^T in binary64 and the bound of the kernels' sums of it.

    Within a block, products of two codes are exact (8 bits) and added in binary32: 128 terms, each sum off by at most
    2^-23 of the sum of magnitudes so far (no rounding mode is assumed).  The block's sum is multiplied by the two scales
    (their product is rounded, 2^-24) and added with one rounding, K / 128 times and once for each wave or piece of K.
    Where the 8-bit matrix instruction adds (wide_sums False), seven of eight consecutive products lose up to 2^-13 of the
    largest of the eight, too."""
    x, w = numbers(xw, xs), numbers(ww, ws, B)
    y = x @ w.T
    env = np.abs(x) @ np.abs(w).T
    blocks = x.shape[1] // B
    bound = env * (128 * 2.0 ** -23 + (blocks + waves + 2) * 2.0 ** -24)
    if not wide_sums:
        k8 = x.shape[1] // 8
        ax, aw = np.abs(x).reshape(-1, k8, 8), np.abs(w).reshape(-1, k8, 8)
        for m in range(0, ax.shape[0], 16):
            bound[m:m + 16] += 7 * 2.0 ** -13 * (ax[m:m + 16, None] * aw[None]).max(3).sum(2)
    return y, bound


def gate(y, bound):
    """silu(gate) * up and its bound: silu' is at most 1.1, |silu(g)| at most |g|; the quotient, the exponential (2 ulp,
    which a factor 1 / (1 + e^-g) takes up to once) and the product round."""
    h = y.shape[1] // 2
    g, u, bg, bu = y[:, :h], y[:, h:], bound[:, :h], bound[:, h:]
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    return s * u, 1.1 * bg * (np.abs(u) + bu) + np.abs(s) * bu + 8 * 2.0 ** -24 * np.abs(s * u)


def check(out, want, bound, what):
    """out: torch tensor; want, bound: binary64 arrays."""
    got = out.detach().float().cpu().numpy().astype(np.float64)
    t = out.dtype
    assert got.shape == want.shape, f"{what}: shape {got.shape}, {want.shape}"
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    if t is torch.float16:  # from 65520 on, half a step past the largest value, the nearest word is an infinity
        high = np.isinf(got) & (np.abs(want) + bound >= 65520) & (np.sign(got) == np.sign(want))
        low = np.isfinite(got) & (np.abs(want) - bound < 65520)
        assert bool((high | low | nan).all()), f"{what}: infinities in other places"
        got = np.where(high, want, got)
    off = np.abs(np.where(nan, 0, got - want))
    most = np.where(nan, 1, bound + HALF[t] * (np.abs(want) + bound) + LEAST[t])
    bad = np.argwhere(off > most)
    assert bad.size == 0, f"{what}: {len(bad)} of {off.size} off, first at {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


def sort(ids, experts):
    """order, places, offsets of int ids [tokens, top], pair by pair."""
    flat = ids.reshape(-1)
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(flat.tolist()):
        if 0 <= e < experts:
            lists[e].append(i)
    order = np.full(flat.size, -1, np.int32)
    places = np.full(flat.size, -1, np.int32)
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    for p, i in enumerate(i for x in lists for i in x):
        order[p] = i
        places[i] = p
    return order, places.reshape(ids.shape), offsets


def few_rows(rows, experts=0):
    """Whether a call's products are exact whatever its output type (include/nq.h states the rule)."""
    return (-(-rows // experts) if experts else rows) <= 16


def experts_product(xw, xs, ww, ws, order, offsets, top, sorted_rows, wide_sums, gated):
    """Each place's product and bound; zeros behind the last place."""
    pairs = order.size
    n = ww.shape[1] // (2 if gated else 1)
    y, bound = np.zeros((pairs, n)), np.zeros((pairs, n))
    for e in range(len(offsets) - 1):
        at = np.arange(offsets[e], offsets[e + 1])
        if at.size == 0:
            continue
        rows = at if sorted_rows else order[at] // top
        v = product(xw[rows], xs[rows], ww[e], ws[e], wide_sums)
        y[at], bound[at] = gate(*v) if gated else v
    return y, bound


def combine(rows, places, weights):
    """Rows back to tokens in binary64, and the bound of binary32 sums: each term one rounding of what is summed so far."""
    t, top = places.shape
    out, env = np.zeros((t, rows.shape[1])), np.zeros((t, rows.shape[1]))
    for c in range(top):
        p = places[:, c]
        live = p >= 0
        term = np.where(live[:, None], rows[np.maximum(p, 0)] * weights[:, c, None], 0)
        out += term
        env += np.abs(term)
    return out, env * top * 2.0 ** -24


def combine_grad(grad, rows, places, weights):
    """Gradients of rows and weights in binary64, and the bound of the second's binary32 sum of `cols` products."""
    g_rows, g_w = np.zeros_like(rows), np.zeros(places.shape)
    bound = np.zeros(places.shape)
    for c in range(places.shape[1]):
        for t in np.nonzero(places[:, c] >= 0)[0]:
            p = places[t, c]
            g_rows[p] = grad[t] * weights[t, c]
            g_w[t, c] = grad[t] @ rows[p]
            bound[t, c] = np.abs(grad[t]) @ np.abs(rows[p]) * (rows.shape[1] + 4) * 2.0 ** -24
    return g_rows, g_w, bound
