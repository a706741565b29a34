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
