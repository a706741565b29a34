"""The attention's launch plan and workspace for the 8-bit key/value cache, on the host (no GPU)."""
import ctypes
import fcntl
import os
import subprocess

import numpy as np
import pytest

import block_quantized_weight_nq_amd as nq

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = os.environ.get("NQ_SANITIZE") == "1"
EMU = os.path.join(HERE, "emu", "libnq_kv_plan_emu_san.so" if SAN else "libnq_kv_plan_emu.so")
CSRC = os.path.join(os.path.dirname(HERE), "block_quantized_weight_nq_amd", "csrc")


@pytest.fixture(scope="module")
def emu():
    src = os.path.join(HERE, "emu", "nq_kv_plan_emu.hip")
    deps = [src] + [os.path.join(CSRC, h) for h in ("nq_kv.h", "nq_decode.h")]
    with open(EMU + ".lock", "w") as lk:
        fcntl.flock(lk, fcntl.LOCK_EX)
        if not os.path.exists(EMU) or any(os.path.getmtime(d) > os.path.getmtime(EMU) for d in deps):
            from emu_lib import SAN_FLAGS
            tmp = f"{EMU}.{os.getpid()}.tmp"
            subprocess.run(["hipcc", "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared",
                            "-fvisibility=hidden", *(SAN_FLAGS if SAN else []), src, "-o", tmp], check=True)
            os.replace(tmp, EMU)
    L = ctypes.CDLL(EMU)
    L.nq_kv_emu_request.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_void_p, ctypes.c_void_p]
    L.nq_kv_emu_call.restype = ctypes.c_long
    L.nq_kv_emu_call.argtypes = ([ctypes.c_void_p] * 2 + [ctypes.c_int] * 10 + [ctypes.c_void_p, ctypes.c_int,
                                 ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p] * 2)
    return L


def find(emu, starts, u, bsh, threads):
    out = np.zeros(2, np.int32)
    r = emu.nq_kv_emu_request(starts.ctypes.data, starts.size - 1, u, bsh, threads, out.ctypes.data, out[1:].ctypes.data)
    return r, int(out[0]), int(out[1])


@pytest.mark.parametrize("requests, threads", [(1, 4), (4, 4), (5, 4), (16, 4), (17, 4), (300, 4), (1000, 16)])
def test_store_finds_the_request_of_each_unit(emu, requests, threads):
    """Every unit's request, as a plain scan of the starts finds it, in rounds that grow with the logarithm."""
    rng = np.random.default_rng(requests)
    for bsh in (4, 7):
        new = rng.choice([0, 0, 1, 15, 16, 17, 200], requests)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        first = (starts >> bsh) + 2 * np.arange(requests + 1)
        for u in range(int(first[-1]) + 3):
            r, bad, rounds = find(emu, starts, u, bsh, threads)
            assert bad == 0 and r == (int(np.searchsorted(first, u, side="right")) - 1 if u < first[-1] else -1)
            assert threads ** rounds <= requests


def test_store_searches_many_requests_in_few_rounds(emu):
    """2^20 and 2^23 requests, 256 threads: at most two rounds before the last."""
    for requests in (1 << 20, (1 << 23) - 1):
        starts = np.arange(requests + 1, dtype=np.int32) // 3
        first = (starts >> 4).astype(np.int64) + 2 * np.arange(requests + 1)
        for r in (0, 1, 255, 256, 65535, 65536, requests // 2, requests - 1):
            assert find(emu, starts, int(first[r]), 4, 256) == (r, 0, 2)


@pytest.mark.parametrize("seed", range(20))
def test_store_search_stays_inside_for_any_starts(emu, seed):
    rng = np.random.default_rng(seed)
    starts = rng.integers(-2 ** 31, 2 ** 31, int(rng.integers(2, 3000))).astype(np.int32)
    for u in list(rng.integers(0, 2 ** 27, 20)) + [0, 1, 2 ** 31]:
        assert find(emu, starts, int(u), 4, 8)[1] == 0


def workspace(tokens, requests, max_new, max_length, heads=8, group=4, dim=128, block=64, window=0, dtype=2):
    """(status, bytes) of nq_kv_attention_workspace."""
    buf = np.zeros(64, np.uint32)
    p = (buf.ctypes.data + 15) // 16 * 16
    d = nq.KvCacheDesc(0, heads, dim, block, 1000, p, p, p, p)
    q_heads, width = heads * group, -(-max_length // block)
    a = nq.KvAttentionArgs(p, q_heads * dim, dim, tokens, q_heads, requests, p, p, p, width, width, window, max_new,
                           max_length, p, 0, dtype, 0.1)
    need = ctypes.c_uint64()
    st = nq.library().nq_kv_attention_workspace(ctypes.byref(d), ctypes.byref(a), ctypes.byref(need))
    return st, need.value


@pytest.mark.parametrize("dim, heads, group", [(64, 8, 1), (128, 8, 4), (256, 4, 4), (128, 1, 8), (128, 2, 40)])
@pytest.mark.parametrize("tokens", [8192, 32768, 131072])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_workspace_of_a_prompt(dim, heads, group, tokens, dtype):
    """A prompt's rows fill the card without being cut, and the kernel for few rows has none of them: the workspace is
    below the output's size."""
    st, need = workspace(tokens, 1, tokens, tokens, heads, group, dim, dtype=dtype)
    assert st == 0 and need <= tokens * heads * group * dim * (4 if dtype == 0 else 2)


@pytest.mark.parametrize("dim, heads, group", [(64, 8, 1), (128, 8, 4), (128, 1, 8)])
def test_workspace_of_a_mixed_step(dim, heads, group):
    """Single tokens beside a prompt: pieces for the tokens that the few-rows kernel can have, not for the prompt's."""
    single = workspace(16, 16, 1, 131072, heads, group, dim)[1]
    few = min(128 // group, 8192)
    st, need = workspace(15 + 8192, 16, 8192, 131072, heads, group, dim)
    assert st == 0 and single > 0 and need <= few * single


def test_sizes_past_the_launch_are_refused():
    """A grid holds less than 2^32 threads along an axis: sizes that need more are refused as such (7), not launched."""
    buf = np.zeros(64, np.uint32)
    p = (buf.ctypes.data + 15) // 16 * 16
    L = nq.library()
    d = nq.KvCacheDesc(0, 1, 64, 16, 1000, p, p, p, p)
    ref = ctypes.byref(d)
    store = lambda tokens, requests: L.nq_kv_store(  # noqa: E731  (no token starts: 1 where the sizes are in order)
        ref, p, 64, 64, p, 64, 64, tokens, 0, p, None, requests, p, None)
    assert store(1, 1 << 23) == 7 and store(31, (1 << 23) - 1) == 1 and store(32, (1 << 23) - 1) == 7
    assert store((1 << 28) - 48, 1) == 1 and store((1 << 28) - 32, 1) == 7
    load = lambda n: L.nq_kv_load(ref, None, n, 0, p, p, None)  # noqa: E731
    assert load((1 << 24) - 1) == 1 and load(1 << 24) == 7
    for heads, group in ((1, 1), (2, 1), (1, 4)):
        most = (1 << 28) // (heads * group)  # its tiles of 16 rows: 2^24 / heads a head
        size = dict(max_length=1 << 16, heads=heads, group=group, dim=64)
        assert workspace(most, 1, most, dtype=0, **size)[0] == 7
        assert workspace(most - 16, 1, most - 16, dtype=0, **size)[0] == 0
        assert workspace(most, 1, most, dtype=1, **size)[0] == 0


# --- a call's plan, pieces and staging --------------------------------------------------------------------------

def run_call(emu, starts, lengths, tokens, heads, group, dim, bsh, dtype, window, max_new, max_length, table, blocks,
             cus=256):
    """(what was wrong, how often each token's row is computed, [splits, splits_few, few_tokens])."""
    rows, cuts = np.zeros(tokens + 1, np.int32), np.zeros(3, np.int32)
    bad = emu.nq_kv_emu_call(starts.ctypes.data, lengths.ctypes.data, lengths.size, tokens, heads, group, dim, bsh, dtype,
                             window, max_new, max_length, table.ctypes.data, table.shape[1], blocks, cus,
                             rows.ctypes.data, cuts.ctypes.data)
    return bad, rows, cuts


def any_table(rng, requests, width, blocks):
    t = rng.integers(0, blocks, (requests, width)).astype(np.int32)
    t[rng.random(t.shape) < 0.1] = rng.choice([-1, -2 ** 31, blocks, 2 ** 31 - 1])
    return t


@pytest.mark.parametrize("dim, heads, group", [(64, 3, 1), (64, 1, 5), (128, 1, 4), (128, 2, 1), (256, 1, 8),
                                               (128, 1, 140)])
@pytest.mark.parametrize("dtype", [0, 2])
@pytest.mark.parametrize("bsh", [4, 7])
def test_a_calls_pieces_and_staging(emu, dim, heads, group, dtype, bsh):
    """The plan that the library makes: no tile or piece beyond its launch, each piece of a row in a place of its own
    inside the workspace, every staged code from its key's own place in the pool, every row within max_new once."""
    rng = np.random.default_rng(dim + group + bsh)
    cut = np.zeros(3, bool)
    for trial in range(12):
        blocks, requests = 7, int(rng.choice([1, 2, 5, 30]))
        if trial == 0:  # one chunk over many keys: cut
            requests = 1
        new = rng.choice([0, 1, 1, 1, 2, 5, 33, 150], requests) if trial else np.array([150])
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        tokens = int(starts[-1]) + int(rng.integers(0, 4)) + (starts[-1] == 0)
        longest = int(rng.choice([64, 700, 3000])) if trial else 3000
        lengths = rng.integers(0 if trial else longest // 2, longest, requests)
        lengths = (lengths + new * (trial % 4 > 0)).astype(np.int32)
        most = int(max(1, new.max()))
        max_new, max_length = most, longest + most
        if trial and trial % 3 == 0:
            max_new, max_length = max(1, most // 2), longest // 2
        window = int(rng.choice([0, 0, 1, 100, 1500])) if trial else 0
        table = any_table(rng, requests, -(-(longest + most) >> bsh) + 1, blocks)
        bad, rows, cuts = run_call(emu, starts, lengths, tokens, heads, group, dim, bsh, dtype, window, max_new,
                                   max_length, table, blocks, cus=int(rng.choice([8, 256])) if trial else 256)
        assert bad == 0, (trial, requests, window, max_new, max_length)
        want = np.zeros(tokens + 1, np.int32)
        for s0, s1 in zip(starts, starts[1:]):
            want[s0:min(s1, s0 + max_new)] = 1
        assert np.array_equal(rows, want)
        cut |= cuts > 1
    assert (cut[1] or group > 128) and (cut[0] or dtype == 0)  # both kernels' rows were cut, where they have some


@pytest.mark.parametrize("seed", range(30))
def test_a_calls_pieces_stay_inside_for_any_lengths(emu, seed):
    """Starts and lengths that no step makes: still nothing outside the workspace, the table or the pool."""
    rng = np.random.default_rng(seed)
    requests, blocks, tokens = int(rng.integers(1, 6)), 5, int(rng.integers(1, 300))
    odd = [-2 ** 31, -1, 0, 1, 7, tokens, tokens + 1, 2 ** 30 + 5, 2 ** 31 - 1]
    starts = rng.choice(odd, requests + 1).astype(np.int32)
    lengths = rng.choice(odd, requests).astype(np.int32)
    # requests that share tokens write their rows' pieces twice: look at one request at a time for that
    for r in range(requests):
        one = np.ascontiguousarray(starts[r:r + 2])
        dim, group = int(rng.choice([64, 128, 256])), int(rng.choice([1, 4, 9]))
        bad, _, _ = run_call(emu, one, lengths[r:r + 1].copy(), tokens, 2, group, dim, 5, int(rng.choice([0, 1])),
                             int(rng.choice([0, 1, 500, 2 ** 30])), int(rng.choice([1, 50, 1 << 20])), 1500,
                             any_table(rng, 1, 40, blocks), blocks)
        assert bad == 0, (one, lengths[r])
