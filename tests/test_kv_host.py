"""The 8-bit key/value cache on the host: argument checks of the C ABI and the binding, and the kernels' index rules
run on the CPU against the buffers (no GPU)."""
import ctypes
import fcntl
import os
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
import kv_ref

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = os.environ.get("NQ_SANITIZE") == "1"
EMU = os.path.join(HERE, "emu", "libnq_kv_emu_san.so" if SAN else "libnq_kv_emu.so")
CSRC = os.path.join(os.path.dirname(HERE), "block_quantized_weight_nq_amd", "csrc")


@pytest.fixture(scope="module")
def emu():
    src = os.path.join(HERE, "emu", "nq_kv_emu.hip")
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
    L.nq_kv_emu_units.restype = ctypes.c_long
    L.nq_kv_emu_units.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                  ctypes.c_void_p]
    L.nq_kv_emu_attention.restype = ctypes.c_long
    L.nq_kv_emu_attention.argtypes = [ctypes.c_int] * 7 + [ctypes.c_void_p] + [ctypes.c_int] * 5 + [ctypes.c_int64,
                                                                                                    ctypes.c_void_p]
    return L


@pytest.mark.parametrize("bsh", [4, 5, 6, 7])
def test_store_units_cover_each_token_once(emu, bsh):
    rng = np.random.default_rng(bsh)
    for trial in range(40):
        R = int(rng.integers(1, 9))
        new = rng.choice([0, 1, 2, (1 << bsh) - 1, 1 << bsh, (1 << bsh) + 1, 5 * (1 << bsh) + 3], R)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        off = rng.integers(0, 1 << bsh, R).astype(np.int32)
        if trial % 3 == 0:
            off[:] = (1 << bsh) - 1
        tokens = int(starts[-1]) + int(rng.integers(0, 5))
        hits = np.zeros(tokens + 1, np.int32)
        assert emu.nq_kv_emu_units(starts.ctypes.data, R, off.ctypes.data, bsh, tokens, hits.ctypes.data) == 0
        assert (hits[: starts[-1]] == 1).all() and (hits[starts[-1]:] == 0).all()


@pytest.mark.parametrize("starts", [[0, -3, 5], [7, 2, 9], [0, 100, 3], [5, 5, 5], [0, 2 ** 31 - 1, 4]])
def test_store_units_stay_inside_for_bad_starts(emu, starts):
    s = np.array(starts, np.int32)
    hits = np.zeros(11, np.int32)
    off = np.array([3, 9], np.int32)
    emu.nq_kv_emu_units(s.ctypes.data, 2, off.ctypes.data, 4, 10, hits.ctypes.data)
    assert hits[10] == 0


@pytest.mark.parametrize("dim, tile", [(64, 64), (128, 64), (128, 32), (256, 32)])
@pytest.mark.parametrize("bsh", [4, 5, 6, 7])
def test_attention_reads_inside_the_pool(emu, dim, tile, bsh):
    """Every address of a launch lies in the pool and every table index in the row, also for tables that name blocks
    outside the pool; the first tile visits each of its keys once."""
    rng = np.random.default_rng(dim + bsh)
    blocks, heads, width = 9, 3, 40
    for trial in range(30):
        table = rng.integers(0, blocks, width).astype(np.int32)
        if trial % 2:
            table[rng.integers(0, width, 12)] = rng.choice([-1, -2 ** 31, blocks, 2 ** 31 - 1], 12)
        cap = int(rng.integers(1, width * (1 << bsh) + 1))
        length = int(rng.choice([0, 1, 15, 16, 17, cap, cap + 100, 2 ** 31 - 1, int(rng.integers(1, cap + 1))]))
        added = int(rng.choice([1, 1, 2, 7, 40]))
        group, window = int(rng.choice([1, 3, 4, 16])), int(rng.choice([0, 0, 1, 50, 1000]))
        chunk = int(rng.choice([512, 576, 1088, 1 << 20]))
        span = min(cap, window + 16 // group + 2 + 63) if window else cap
        splits = -(-span // chunk)
        visits = np.zeros(cap + 1, np.int32)
        bad = emu.nq_kv_emu_attention(added, length, cap, group, window, chunk, splits, table.ctypes.data, width, bsh,
                                      dim, tile, heads, blocks, visits.ctypes.data)
        assert bad == 0, (trial, length, cap, added, group, window, chunk)
        last = min((min(16, added * group) - 1) // group, added - 1)
        end = max(0, min(length, cap, length - added + last + 1))
        beg = max(0, min(end, length - added - window + 1)) if window else 0
        want = np.zeros(cap + 1, np.int32)
        for key in range(beg, end):
            want[key] = 0 <= table[key >> bsh] < blocks
        assert np.array_equal(visits, want)


# --- refusals ---------------------------------------------------------------------------------------------------

def _cache(**kw):
    buf = np.zeros(64, np.uint32)
    p = (buf.ctypes.data + 15) // 16 * 16
    c = dict(code=0, heads=2, dim=128, block=16, blocks=4, k=p, v=p, k_scale=p, v_scale=p)
    c.update(kw)
    d = nq.KvCacheDesc(*c.values())
    d._keep = buf
    return d, p


def _load(d, n=1, dtype=0, ids=64, k=64, v=64):
    return nq.library().nq_kv_load(ctypes.byref(d), ids, n, dtype, k, v, None)


@pytest.mark.parametrize("kw, status", [
    (dict(code=2), 2), (dict(code=-1), 2), (dict(dim=0), 4), (dict(dim=96), 4), (dict(dim=512), 4), (dict(block=8), 4),
    (dict(block=48), 4), (dict(block=256), 4), (dict(heads=0), 4), (dict(heads=65536), 4), (dict(blocks=0), 4),
    (dict(blocks=2 ** 31), 4), (dict(k=0), 1), (dict(v=0), 1), (dict(k_scale=0), 1), (dict(v_scale=0), 1),
    (dict(k=72), 11), (dict(v=72), 11), (dict(k_scale=66), 11), (dict(v_scale=66), 11)])
def test_every_call_checks_the_cache(kw, status):
    d, p = _cache(**kw)
    L, ref = nq.library(), ctypes.byref(d)
    assert _load(d) == status
    assert L.nq_kv_store(ref, p, 256, 128, p, 256, 128, 1, 0, p, p, 1, p, None) == status
    args = nq.KvAttentionArgs(p, 256, 128, 1, 2, 1, p, p, p, 1, 1, 0, 1, 16, p, p, 0, 1.0)
    need = ctypes.c_uint64(7)
    assert L.nq_kv_attention_workspace(ref, ctypes.byref(args), ctypes.byref(need)) == status and need.value == 0
    assert L.nq_kv_attention(ref, ctypes.byref(args), None, 0, None) == status


def test_null_cache_and_arguments():
    L = nq.library()
    d, p = _cache()
    need = ctypes.c_uint64()
    assert L.nq_kv_load(None, p, 1, 0, p, p, None) == 1
    assert L.nq_kv_attention_workspace(ctypes.byref(d), None, ctypes.byref(need)) == 1
    assert L.nq_kv_attention_workspace(ctypes.byref(d), None, None) == 1
    assert L.nq_kv_attention(None, None, None, 0, None) == 1


def test_load_refusals():
    d, _ = _cache()
    assert _load(d, n=0, ids=0, k=0, v=0) == 0
    assert _load(d, n=-1) == 4
    assert _load(d, n=2 ** 31) == 7
    assert _load(d, dtype=3) == 8 and _load(d, dtype=-1) == 8
    assert _load(d, ids=0) == 1 and _load(d, k=0) == 1 and _load(d, v=0) == 1
    assert _load(d, ids=66) == 11 and _load(d, k=72) == 11 and _load(d, v=68) == 11


def test_store_refusals():
    d, p = _cache()
    base = dict(k=p, kt=256, kh=128, v=p, vt=256, vh=128, tokens=1, dtype=0, slots=p, starts=p, requests=1, status=p)

    def call(**kw):
        a = dict(base, **kw)
        return nq.library().nq_kv_store(ctypes.byref(d), *a.values(), None)

    assert call(dtype=3) == 8 and call(dtype=-1) == 8
    assert call(tokens=-1) == 4 and call(requests=0) == 4
    assert call(tokens=2 ** 31) == 7 and call(requests=2 ** 24) == 7
    for s in ("kt", "vt", "kh", "vh"):
        assert call(**{s: -1}) == 7 and call(**{s: 2 ** 61}) == 7
    for s in ("k", "v", "slots", "starts", "status"):
        assert call(**{s: 0}) == 1
    assert call(k=p + 2) == 11 and call(v=p + 1, dtype=2) == 11 and call(slots=p + 4) == 11
    assert call(starts=p + 2) == 11 and call(status=p + 1) == 11


def test_tables_refusals():
    p = (np.zeros(64, np.uint32).ctypes.data + 15) // 16 * 16
    base = dict(lengths=p, added=p, requests=2, table=p, width=4, stride=4, ring=p, ring_size=8, state=p, block=16,
                tokens=4, lengths_out=p, starts=p, slots=p, state_out=p, status=p)

    def call(**kw):
        return nq.library().nq_kv_tables(*dict(base, **kw).values(), None)

    for bad in (dict(block=0), dict(block=24), dict(block=256), dict(requests=0), dict(requests=2 ** 20), dict(width=0),
                dict(ring_size=0), dict(tokens=-1), dict(stride=3)):
        assert call(**bad) == 4, bad
    for bad in (dict(width=2 ** 31), dict(ring_size=2 ** 31), dict(tokens=2 ** 31), dict(stride=-4), dict(stride=2 ** 61)):
        assert call(**bad) == 7, bad
    for s in ("lengths", "added", "table", "ring", "state", "lengths_out", "starts", "slots", "state_out", "status"):
        assert call(**{s: 0}) == 1, s
        assert call(**{s: p + (4 if s == "slots" else 2)}) == 11, s


def test_attention_refusals_and_workspace():
    d, p = _cache()
    base = dict(q=p, qt=256, qh=128, tokens=1, q_heads=4, requests=1, starts=p, lengths=p, table=p, width=8, stride=8,
                window=0, max_new=1, max_length=128, out=p, lse=0, dtype=2, scale=0.1)

    def call(ws=None, ws_bytes=0, **kw):
        a = nq.KvAttentionArgs(*dict(base, **kw).values())
        return nq.library().nq_kv_attention(ctypes.byref(d), ctypes.byref(a), ws, ws_bytes, None)

    def need(**kw):
        a, n = nq.KvAttentionArgs(*dict(base, **kw).values()), ctypes.c_uint64()
        assert nq.library().nq_kv_attention_workspace(ctypes.byref(d), ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    for bad in (dict(tokens=-1), dict(q_heads=0), dict(q_heads=3), dict(requests=0), dict(requests=65535),
                dict(max_new=0), dict(max_length=0), dict(window=-1), dict(width=0), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert call(**bad) == 4, bad
    for bad in (dict(q_heads=2 ** 16), dict(tokens=2 ** 29), dict(max_new=2 ** 31), dict(max_length=2 ** 31),
                dict(window=2 ** 31), dict(width=2 ** 31), dict(stride=-1), dict(qt=-1), dict(qh=-1), dict(qt=2 ** 61)):
        assert call(**bad) == 7, bad
    assert call(dtype=3) == 8
    for s in ("q", "starts", "lengths", "table", "out"):
        assert call(**{s: 0}) == 1, s
    for s, at in (("q", 1), ("starts", 2), ("lengths", 2), ("table", 2), ("out", 8), ("lse", 2)):
        assert call(**{s: p + at}) == 11, s
    assert need() == 0
    long = dict(width=10 ** 5, stride=10 ** 5, max_length=10 ** 6)
    assert need(**long) > 0
    assert call(**long) == 12
    assert call(ws=p, ws_bytes=need(**long) - 1, **long) == 12
    assert call(ws=p + 8, ws_bytes=need(**long), **long) == 11
    assert need(tokens=0, **long) == 0 and call(tokens=0, q=0, out=0, **long) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros((2, 1, 16, 64), dtype=torch.int8)
    v, s = torch.zeros((2, 1, 64, 16), dtype=torch.int8), torch.zeros((2, 1))
    with pytest.raises(ValueError, match="CUDA"):
        nq.KvCache(k, v, s, s)
    with pytest.raises(ValueError, match="int8"):
        nq.KvCache(k.float(), v.float(), s, s)
    with pytest.raises(ValueError, match="int8"):
        nq.KvCache(k, v.view(torch.float8_e4m3fn), s, s)
    with pytest.raises(ValueError, match="dim"):
        nq.KvCache(k, k, s, s)
    with pytest.raises(ValueError, match="dim"):
        nq.KvCache(k[0], v[0], s, s)
    with pytest.raises(ValueError, match="block"):
        nq.KvCache(k[:, :, :8].contiguous(), v[..., :8].contiguous(), s, s)
    with pytest.raises(ValueError, match="scales"):
        nq.KvCache(k, v, s, s.double())
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nq.kv_tables(i, i, i.view(4, 1), i, i[:2], 16, 4)


# --- the reference itself ---------------------------------------------------------------------------------------

def test_reference_codes():
    """The E4M3 grid and nearest rule against torch's conversion, and the tables' reference on a hand-made step."""
    w = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(w, kv_ref.E4M3.astype(np.float32), equal_nan=True)
    x = np.random.default_rng(0).normal(0, 100, 20000).astype(np.float32)
    x[:2000] *= 1e-4
    x[2000:2254] = np.r_[kv_ref.E4M3[:127], -kv_ref.E4M3[:127]] * np.float32(1.0625)
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_ref.to_codes(x, "e4m3"), want)
    ring = np.array([7, 8, 9, 3], np.int32)
    t, ring, out, starts, slots, state, st = kv_ref.tables(
        np.array([15, 16, 20], np.int32), np.array([2, 0, -1], np.int32),
        np.array([[1, -1], [2, -1], [4, 5]], np.int32), ring, [1, 2], 16, 4)
    assert st == 0 and out.tolist() == [17, 16, 0] and starts.tolist() == [0, 2, 2, 2]
    assert t.tolist() == [[1, 8], [2, -1], [4, 5]] and slots.tolist() == [31, 128, -1, -1]
    assert ring.tolist() == [5, 8, 9, 4] and state.tolist() == [2, 3]
