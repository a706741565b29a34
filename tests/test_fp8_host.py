"""E4M3 blocks and the experts' rows on the host: argument checks of the C ABI, the binding's devices and streams, the
launch plan and the tile rule against the tensors (no GPU)."""
import ctypes
import fcntl
import os
import subprocess
import types

import numpy as np
import pytest
import torch

import block_quantized_weight_nq_amd as nq
from test_binding_device import Tensor, gpus  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = os.environ.get("NQ_SANITIZE") == "1"
EMU = os.path.join(HERE, "emu", "libnq_fp8_emu_san.so" if SAN else "libnq_fp8_emu.so")
CSRC = os.path.join(os.path.dirname(HERE), "block_quantized_weight_nq_amd", "csrc")
P = 1 << 20  # an aligned address that no refused call reads


# --- refusals ---------------------------------------------------------------------------------------------------

def quantize(x=P, dtype=0, matrices=1, rows=4, cols=256, stride=256, tile=1, codes=P, scales=P):
    return nq.library().nq_quantize_fp8_block(x, dtype, matrices, rows, cols, stride, tile, codes, scales, None)


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), 8), (dict(dtype=-1), 8), (dict(rows=-1), 4), (dict(cols=-128), 4), (dict(matrices=-1), 4), (dict(tile=64), 4),
    (dict(tile=0), 4), (dict(cols=100), 5), (dict(cols=200, rows=0), 5), (dict(rows=2 ** 30 + 1), 7), (dict(cols=2 ** 31), 7),
    (dict(rows=2 ** 30, cols=2 ** 30), 7), (dict(matrices=2 ** 30, rows=2 ** 30), 7), (dict(stride=-1), 4),
    (dict(stride=2 ** 60), 7), (dict(x=0), 1), (dict(codes=0), 1), (dict(scales=0), 1), (dict(x=P + 2), 11), (dict(dtype=2, x=P + 1), 11),
    (dict(codes=P + 8), 11), (dict(scales=P + 2), 11), (dict(rows=0, x=0, codes=0, scales=0), 0), (dict(cols=0, x=0), 0)])
def test_quantize_refuses(kw, status):
    assert quantize(**kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), 8), (dict(rows=-1), 4), (dict(cols=130), 5), (dict(tile=2), 4), (dict(rows=2 ** 31), 7), (dict(codes=0), 1),
    (dict(scales=0), 1), (dict(out=0), 1), (dict(codes=P + 4), 11), (dict(scales=P + 1), 11), (dict(out=P + 8), 11), (dict(rows=0, out=0), 0)])
def test_values_refuse(kw, status):
    a = dict(codes=P, scales=P, matrices=1, rows=4, cols=256, tile=1, dtype=0, out=P)
    a.update(kw)
    assert nq.library().nq_dequantize_fp8_block(*a.values(), None) == status


ARGS = dict(x=P, x_row_stride=256, x_scales=0, weight=P, weight_scales=P, out=P, rows=4, N=512, K=256, x_dtype=2, out_dtype=2,
            gated=0, sorted=0)
PLAN = dict(order=P, places=P, offsets=P, tokens=4, top=2, experts=8)


def product(plan=None, ws=0, ws_bytes=0, asked=False, **kw):
    args = nq.Fp8BlockArgs(*{**ARGS, **kw}.values())
    plan = ctypes.byref(nq.MoePlanDesc(*{**PLAN, **plan}.values())) if plan is not None else None
    need = ctypes.c_uint64(77)
    L = nq.library()
    st = L.nq_gemm_fp8_block_workspace(ctypes.byref(args), plan, need)
    assert st == 0 or need.value == 0
    if asked:
        return st, need.value
    return L.nq_gemm_fp8_block(ctypes.byref(args), plan, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, status", [
    (dict(x_dtype=3), 8), (dict(out_dtype=3), 8), (dict(out_dtype=-1), 8), (dict(rows=-1), 4), (dict(N=0), 4), (dict(K=0), 4),
    (dict(gated=2), 4), (dict(sorted=1), 4), (dict(K=192), 5), (dict(gated=1, N=384), 5), (dict(rows=2 ** 30 + 1), 7),
    (dict(N=2 ** 31), 7), (dict(K=2 ** 31), 7), (dict(x_row_stride=-1), 4), (dict(x_row_stride=2 ** 60), 7),
    (dict(rows=2 ** 30, N=2 ** 30), 7), (dict(x_scales=P, x_row_stride=264), 11)])
def test_product_and_workspace_refuse(kw, status):
    assert product(asked=True, **kw) == (status, 0)
    assert product(**kw) == status


@pytest.mark.parametrize("kw, status", [
    (dict(x=0), 1), (dict(weight=0), 1), (dict(weight_scales=0), 1), (dict(out=0), 1), (dict(x=P + 1), 11), (dict(weight=P + 8), 11),
    (dict(weight_scales=P + 2), 11), (dict(out=P + 4), 11), (dict(x_scales=P + 2), 11), (dict(x_scales=P, x=P + 8), 11),
    (dict(ws=P + 8), 11), (dict(rows=300), 12), (dict(rows=300, ws=P, ws_bytes=4096), 12), (dict(rows=0, x=0, out=0), 0)])
def test_product_refuses_pointers_and_workspace(kw, status):
    assert product(**kw) == status


@pytest.mark.parametrize("plan, kw, status", [
    (dict(), dict(rows=5), 4), (dict(), dict(sorted=1), 4), (dict(tokens=-1), {}, 4), (dict(top=0), {}, 4), (dict(experts=0), {}, 4),
    (dict(experts=1025), {}, 7), (dict(tokens=2 ** 29, top=4), {}, 7), (dict(top=1025), {}, 7), (dict(offsets=0), {}, 1), (dict(order=0), {}, 1),
    (dict(places=0), {}, 1), (dict(order=P + 2), {}, 11), (dict(offsets=P + 1), {}, 11)])
def test_product_refuses_plans(plan, kw, status):
    assert product(plan=plan, **kw) == status
    assert product(plan=plan, asked=True, **kw)[0] == status


def test_empty_plan_launches_nothing():
    assert product(plan=dict(tokens=0, order=0, places=0), rows=0, x=0, out=0) == 0


@pytest.mark.parametrize("kw, status", [
    (dict(tokens=-1), 4), (dict(top=0), 4), (dict(experts=0), 4), (dict(experts=1025), 7), (dict(tokens=2 ** 30, top=2), 7),
    (dict(tokens=1, top=1025), 7), (dict(wide=2), 8), (dict(ids=0), 1), (dict(order=0), 1), (dict(places=0), 1), (dict(offsets=0), 1), (dict(ids=P + 4, wide=1), 11),
    (dict(ids=P + 2), 11), (dict(order=P + 2), 11), (dict(ws=P + 1), 11), (dict(tokens=5000), 12), (dict(tokens=5000, ws=P, ws_bytes=12), 12)])
def test_sort_refuses(kw, status):
    a = dict(ids=P, wide=0, tokens=9, top=2, experts=8, order=P, places=P, offsets=P, ws=0, ws_bytes=0)
    a.update(kw)
    assert nq.library().nq_moe_sort(*a.values(), None) == status


@pytest.mark.parametrize("tokens, top, chunks", [(4096, 1, 0), (4097, 1, 2), (2 ** 18, 8, 512), (2 ** 18 + 1, 8, 257), (2 ** 30, 1, 512), (2 ** 20 + 1, 1023, 512)])
def test_sort_workspace_stays_small(tokens, top, chunks):
    """At most 512 workgroups, each of which reads the counts of all."""
    need = ctypes.c_uint64()
    assert nq.library().nq_moe_sort_workspace(tokens, top, 96, ctypes.byref(need)) == 0
    assert need.value == chunks * 96 * 4


@pytest.mark.parametrize("plan, kw, status", [
    ({}, dict(dtype=3), 8), ({}, dict(cols=-1), 4), ({}, dict(cols=2 ** 31), 7), ({}, dict(stride=-1), 4), ({}, dict(stride=2 ** 60), 7),
    ({}, dict(rows=0), 1), ({}, dict(out=0), 1), ({}, dict(rows=P + 2), 11), ({}, dict(weights=P + 2), 11), ({}, dict(out=P + 1), 11),
    (dict(tokens=0, order=0, places=0), {}, 0), ({}, dict(cols=0), 0), (dict(places=0), {}, 1)])
def test_combine_refuses(plan, kw, status):
    d = nq.MoePlanDesc(*{**PLAN, **plan}.values())
    a = dict(rows=P, stride=64, dtype=0, cols=64, weights=P, out=P)
    a.update(kw)
    L = nq.library()
    assert L.nq_moe_combine(ctypes.byref(d), *a.values(), None) == status
    if not kw.get("cols") == 0:
        st = L.nq_moe_combine_grad(ctypes.byref(d), P, a["stride"], a["rows"], a["stride"], a["dtype"], a["cols"], a["weights"],
                                   a["out"], P, None)
        assert st == status


@pytest.mark.parametrize("plan, kw, status", [
    ({}, dict(nbytes=-1), 4), ({}, dict(nbytes=2 ** 33), 7), ({}, dict(stride=-4), 4), ({}, dict(x=0), 1), ({}, dict(out=0), 1),
    ({}, dict(nbytes=0, x=0), 0), (dict(experts=0), {}, 4)])
def test_gather_refuses(plan, kw, status):
    d = nq.MoePlanDesc(*{**PLAN, **plan}.values())
    a = dict(x=P, nbytes=64, stride=64, out=P)
    a.update(kw)
    assert nq.library().nq_moe_gather(ctypes.byref(d), *a.values(), None) == status


def test_null_arguments():
    L = nq.library()
    need = ctypes.c_uint64(5)
    assert L.nq_gemm_fp8_block_workspace(None, None, need) == 1 and need.value == 0
    assert L.nq_gemm_fp8_block(None, None, None, 0, None) == 1
    assert L.nq_moe_sort_workspace(1, 1, 1, None) == 1
    assert L.nq_moe_gather(None, P, 4, 4, P, None) == 1
    assert L.nq_moe_combine(None, P, 4, 0, 4, None, P, None) == 1


# --- the binding ------------------------------------------------------------------------------------------------

def block_calls(index):
    f8 = lambda *shape: Tensor(shape, torch.float8_e4m3fn, index)  # noqa: E731
    f32 = lambda *shape: Tensor(shape, torch.float32, index)  # noqa: E731
    i32 = lambda *shape: Tensor(shape, torch.int32, index)  # noqa: E731
    one, many = nq.Fp8Weight(f8(256, 128), f32(2, 1)), nq.Fp8Weight(f8(4, 256, 128), f32(4, 2, 1))
    plan = nq.MoePlan(i32(6), i32(3, 2), i32(5))
    x = Tensor((3, 128), torch.bfloat16, index)
    rows = f32(6, 8)
    return [
        lambda **kw: nq.quantize_fp8_block(x, **kw), lambda **kw: nq.dequantize_fp8_block(f8(3, 128), f32(3, 1), **kw),
        lambda **kw: nq.gemm_fp8_block(one, x, **kw), lambda **kw: nq.moe_gemm_fp8_block(many, x, plan, **kw),
        lambda **kw: nq.moe_gather(x, plan, **kw), lambda **kw: nq.moe_combine(rows, plan, f32(3, 2), **kw),
        lambda **kw: nq.moe_combine_grad(f32(3, 8), rows, plan, f32(3, 2), **kw)]


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_their_tensors_device(gpus, index):  # noqa: F811
    Tensor.element_size = lambda self: 4
    for call in block_calls(index):
        gpus.calls.clear()
        call()
        assert gpus.calls and all(device == index for _, device in gpus.calls), gpus.calls
        assert gpus.device == 0


def test_a_stream_is_of_the_tensors_device(gpus):  # noqa: F811
    Tensor.element_size = lambda self: 4
    for call in block_calls(1):
        gpus.calls.clear()
        call(stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
        assert gpus.calls and all(device == 1 for _, device in gpus.calls)
        gpus.calls.clear()
        with pytest.raises(ValueError, match="stream"):
            call(stream=types.SimpleNamespace(device=torch.device("cuda", 0)))
        assert not gpus.calls and gpus.device == 0


# --- the tile rule ----------------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def emu():
    src = os.path.join(HERE, "emu", "nq_fp8_emu.hip")
    deps = [src, os.path.join(CSRC, "nq_fp8b.h")]
    with open(EMU + ".lock", "w") as lk:
        fcntl.flock(lk, fcntl.LOCK_EX)
        if not os.path.exists(EMU) or any(os.path.getmtime(d) > os.path.getmtime(EMU) for d in deps):
            from emu_lib import SAN_FLAGS
            tmp = f"{EMU}.{os.getpid()}.tmp"
            subprocess.run(["hipcc", "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared",
                            "-fvisibility=hidden", *(SAN_FLAGS if SAN else []), src, "-o", tmp], check=True)
            os.replace(tmp, EMU)
    L = ctypes.CDLL(EMU)
    L.nq_fp8_emu_tiles.restype = ctypes.c_int64
    L.nq_fp8_emu_tiles.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    L.nq_fp8_emu_plan.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int] * 5 + [ctypes.c_int64, ctypes.c_void_p]
    L.nq_fp8_emu_plan.restype = None
    L.nq_fp8_emu_grid.restype = ctypes.c_int64
    L.nq_fp8_emu_grid.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
    return L


def tiles(emu, offsets, rows, bm):
    """How often each row is in a tile and of which expert; -1 is behind the last."""
    hits, expert = np.zeros(rows + 1, np.int32), np.full(rows + 1, -9, np.int32)
    o = np.array(offsets, np.int32)
    bad = emu.nq_fp8_emu_tiles(o.ctypes.data, o.size - 1, rows, bm, hits.ctypes.data, expert.ctypes.data)
    return bad, hits, expert


@pytest.mark.parametrize("bm", [16, 32, 64, 128, 256])
def test_tiles_cover_each_row_once(emu, bm):
    rng = np.random.default_rng(bm)
    for trial in range(60):
        experts = int(rng.choice([1, 2, 5, 63, 64, 65, 200]))
        counts = rng.choice([0, 0, 1, bm - 1, bm, bm + 1, 3 * bm + 5], experts)
        offsets = np.concatenate([[0], np.cumsum(counts)])
        rows = int(offsets[-1]) + int(rng.choice([0, 0, 1, bm, 2 * bm + 3]))
        if rows == 0:
            continue
        bad, hits, expert = tiles(emu, offsets, rows, bm)
        assert bad == 0 and (hits[:rows] == 1).all() and hits[rows] == 0
        want = np.repeat(np.arange(experts), counts)
        assert np.array_equal(expert[: offsets[-1]], want) and (expert[offsets[-1]:rows] == -1).all()


def test_tiles_of_any_offsets_stay_inside(emu):
    rng = np.random.default_rng(0)
    for trial in range(300):
        experts, rows = int(rng.choice([1, 3, 64, 70])), int(rng.choice([1, 17, 300]))
        offsets = rng.choice([-2 ** 31, -5, 0, 1, rows - 1, rows, rows + 1, 2 ** 31 - 1], experts + 1)
        assert tiles(emu, offsets, rows, int(rng.choice([16, 64, 256])))[0] == 0


# --- the plan ---------------------------------------------------------------------------------------------------

PLAN_NAMES = ("few weight_tiles config waves splits per_split quantize tiles_m codes scales part chunk depth").split()


def plan(emu, x_rows, rows, experts, N, K, gated=0, codes=0, raw=1, wide=0, far=0, cus=256):
    out = np.zeros(len(PLAN_NAMES), np.int64)
    emu.nq_fp8_emu_plan(x_rows, rows, experts, N, K, gated, codes, raw, wide, far, cus, out.ctypes.data)
    return types.SimpleNamespace(**dict(zip(PLAN_NAMES, out.tolist())))


def test_plans_cover_the_product(emu):
    """Pieces of K, row tiles, LDS and workspace of plans over the range of sizes."""
    rng = np.random.default_rng(1)
    for trial in range(3000):
        experts = int(rng.choice([0, 0, 1, 7, 64, 256, 1024]))
        top = int(rng.choice([1, 2, 8])) if experts else 1
        tokens = int(np.exp(rng.uniform(0, np.log(2e5))))
        rows, K = tokens * top, 128 * int(np.exp(rng.uniform(0, np.log(256))))
        N = int(np.exp(rng.uniform(0, np.log(4e4))))
        gated, codes, raw, wide, far = (int(rng.integers(0, 2)) for _ in range(5))
        N = max(256, N // 256 * 256) if gated else N
        x_rows = rows if rng.integers(0, 2) else tokens
        p = plan(emu, x_rows, rows, experts, N, K, gated, codes, raw, wide, far)
        KB = K // 128
        assert p.few == ((-(-rows // experts) if experts else rows) <= 16)
        assert (p.splits - 1) * p.per_split < KB <= p.splits * p.per_split
        assert p.splits == 1 or (not experts and not p.few)
        bm = 16 if p.few else (64, 128, 256, 128, 64, 128)[p.config]
        assert p.tiles_m >= -(-rows // bm) and (experts == 0 or p.tiles_m <= rows)
        assert p.part == (-(-p.splits * rows * N * 4 // 256) * 256 if p.splits > 1 else 0)
        assert (p.codes > 0) == (p.scales > 0) == bool(p.quantize) and p.codes >= p.quantize * x_rows * K
        assert p.scales >= p.quantize * x_rows * KB * 4 and p.codes % 256 == p.scales % 256 == 0
        assert not (codes and p.quantize) and (raw or codes or p.quantize)
        if p.few:
            assert 1 <= p.waves <= 8 and p.waves <= KB and p.weight_tiles in ((2, 4) if gated else (1, 2))
            assert p.chunk % (p.depth * p.waves) == 0 and p.chunk > 0
            assert max(p.chunk * min(rows, 16) * 132, p.waves * p.weight_tiles * 1024) <= 65536
        else:
            assert p.config not in (0, 3) or p.per_split <= 32
            assert (p.config == 5) == bool(far if codes else x_rows * K > 2 ** 32) and not (wide and p.config == 2)


def test_grids_have_each_tile_once(emu):
    rng = np.random.default_rng(2)
    for trial in range(400):
        m, n = int(np.exp(rng.uniform(0, np.log(400)))), int(np.exp(rng.uniform(0, np.log(200))))
        hits = np.zeros(m * n, np.int32)
        assert emu.nq_fp8_emu_grid(m, n, hits.ctypes.data) == 0
        assert (hits == 1).all(), (m, n)


# --- types ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.float64, torch.uint8, torch.float8_e5m2])
def test_types_that_no_call_takes_are_refused_as_such(gpus, monkeypatch, dtype):  # noqa: F811
    """NQ_ERR_BAD_DTYPE of the library itself, for inputs and outputs alike."""
    monkeypatch.setattr(nq, "_LIB", None)
    f8 = lambda *shape: Tensor(shape, torch.float8_e4m3fn, 0)  # noqa: E731
    f32 = lambda *shape: Tensor(shape, torch.float32, 0)  # noqa: E731
    i32 = lambda *shape: Tensor(shape, torch.int32, 0)  # noqa: E731
    one, many = nq.Fp8Weight(f8(256, 128), f32(2, 1)), nq.Fp8Weight(f8(4, 256, 128), f32(4, 2, 1))
    plan = nq.MoePlan(i32(6), i32(3, 2), i32(5))
    x, other, rows = f32(3, 128), Tensor((3, 128), dtype, 0), Tensor((6, 8), dtype, 0)
    for call in (lambda: nq.quantize_fp8_block(other), lambda: nq.quantize_fp8_block(Tensor((2, 3, 128), dtype, 0), 128),
                 lambda: nq.dequantize_fp8_block(f8(3, 128), f32(3, 1), out_dtype=dtype), lambda: nq.gemm_fp8_block(one, other),
                 lambda: nq.gemm_fp8_block(one, x, out_dtype=dtype), lambda: nq.gemm_fp8_block(one, f8(3, 128), f32(3, 1), out_dtype=dtype),
                 lambda: nq.moe_gemm_fp8_block(many, other, plan), lambda: nq.moe_gemm_fp8_block(many, x, plan, out_dtype=dtype),
                 lambda: nq.moe_combine(rows, plan), lambda: nq.moe_combine_grad(Tensor((3, 8), dtype, 0), rows, plan),
                 lambda: nq.gemm_fp8_block(one, f8(3, 128))):  # codes without their scales
        with pytest.raises(nq.NqError) as refused:
            call()
        assert refused.value.status == 8


# --- the wave's search of a tile --------------------------------------------------------------------------------

def search(emu, offsets, rows, bm, t):
    """What the kernels' wave finds for tile t, and what the rule says: (expert, first, count) each."""
    o, found, rule = np.array(offsets, np.int32), np.zeros(3, np.int64), np.zeros(3, np.int64)
    emu.nq_fp8_emu_search.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
    emu.nq_fp8_emu_search(o.ctypes.data, o.size - 1, rows, bm, t, found.ctypes.data, rule.ctypes.data)
    return found.tolist(), rule.tolist()


@pytest.mark.parametrize("bm", [16, 64, 128, 256])
def test_the_waves_search_follows_the_rule(emu, bm):
    """Every tile of offsets that a sort gives, and those past the last."""
    rng = np.random.default_rng(bm)
    for trial in range(60):
        experts = int(rng.choice([1, 2, 5, 62, 63, 64, 65, 127, 128, 200, 1024]))
        counts = rng.choice([0, 0, 1, bm - 1, bm, bm + 1, 3 * bm + 5], experts)
        offsets = np.concatenate([[0], np.cumsum(counts)])
        rows = int(offsets[-1]) + int(rng.choice([0, 0, 1, bm, 2 * bm + 3]))
        tiles = int(sum(-(-c // bm) for c in counts)) + -(-(rows - int(offsets[-1])) // bm)
        for t in range(tiles + 3) if tiles < 60 else np.unique(np.r_[0, tiles - 1, tiles, tiles + 2, rng.integers(0, tiles, 40)]):
            found, rule = search(emu, offsets, rows, bm, int(t))
            assert found == rule if t < tiles else found[2] == rule[2] == 0, (experts, rows, t)
    # many rows of one expert, and 2^30 rows
    for offsets, rows in (([0, 2 ** 30], 2 ** 30), ([0] * 900 + [2 ** 30] * 124, 2 ** 30), ([0, 5, 2 ** 30 - 7], 2 ** 30)):
        for t in np.r_[0, 1, 2 ** 30 // bm - 1, 2 ** 30 // bm, 2 ** 30 // bm + 2, rng.integers(0, 2 ** 30 // bm, 20)]:
            found, rule = search(emu, offsets, rows, bm, int(t))
            assert found == rule or (found[2] == rule[2] == 0), (rows, t)


def test_the_waves_search_of_any_offsets_stays_inside(emu):
    """Offsets that no sort gives, sums past 32 bits among them: a tile lies within the rows, and within what its expert's
    offsets say of them."""
    rng = np.random.default_rng(1)
    for trial in range(4000):
        experts, rows = int(rng.choice([1, 3, 63, 64, 70, 300, 1024])), int(rng.choice([1, 17, 300, 2 ** 20 + 3, 2 ** 30]))
        bm = int(rng.choice([16, 64, 128, 256]))
        offsets = rng.choice([-2 ** 31, -5, 0, 1, rows // 2, rows - 1, rows, min(rows + 1, 2 ** 31 - 1), 2 ** 31 - 1], experts + 1)
        if trial % 3 == 0:  # from 0 to all rows and back: every second segment has them all
            offsets = np.arange(experts + 1) % 2 * rows
        t = int(rng.choice([0, 1, 7, rows // bm, rows // bm + experts, 2 ** 26, 2 ** 31 - 1]))
        (e, first, count), _ = search(emu, offsets, rows, bm, t)
        assert 0 <= count <= bm and -1 <= e < experts
        if count:
            lo = np.clip(offsets[e if e >= 0 else experts], 0, rows)
            hi = np.clip(offsets[e + 1], 0, rows) if e >= 0 else rows
            assert lo <= first and first + count <= hi <= rows, (offsets[:8], rows, bm, t)


# --- what the GPU tests reach -----------------------------------------------------------------------------------

def test_the_sizes_of_the_gpu_tests_reach_every_instance(emu):
    """On 256 compute units, which an MI355X has: every tile and form of the many-rows kernel that the plan can choose, each in
    pieces too where it can be, with more than sixteen blocks of K in a piece (scales of two places in turn where there are
    two buffers, both halves of them where there are four); the few-rows kernel with each number of weight tiles, and with
    codes in LDS that are replaced."""
    from fp8_cases import EXPERTS, FAR, FAR_EXPERTS, FEW, FEW_EXPERTS, PRODUCTS
    seen, pieces, odd = set(), set(), set()
    for far, one, several in ((0, PRODUCTS, EXPERTS), (1, FAR, FAR_EXPERTS)):
        for m, n, kb, gated, wide in one:
            p = plan(emu, m, m, 0, n, 128 * kb, gated, far, 1, wide, far)
            key = (p.config, "one", gated, wide)
            assert not p.few
            if p.per_split > 16:
                (seen if p.splits == 1 else pieces).add(key)
            if p.per_split > 16 and p.per_split % 2:
                odd.add(key)
        for tokens, top, experts, n, kb, gated, wide in several:
            p = plan(emu, tokens, tokens * top, experts, n, 128 * kb, gated, far, 1, wide, far)
            assert not p.few
            if p.per_split > 16:
                seen.add((p.config, "experts", gated, wide))
    every = {(c, kind, g, w) for c in range(6) for kind in ("one", "experts") for g in (0, 1) for w in (0, 1) if not (c == 2 and w)}
    assert seen == every
    assert pieces >= {k for k in every if k[1] == "one" and k[0] != 5}
    assert odd >= {k for k in every if k[1] == "one" and k[0] in (1, 2, 4, 5)}
    tiles, refilled = set(), set()
    for m, n, kb, gated in FEW:
        p = plan(emu, m, m, 0, n, 128 * kb, gated)
        tiles.add((p.weight_tiles, gated, "values" if not p.quantize else "codes"))
        refilled.add(p.few and not p.quantize and kb > p.chunk and ("one", kb % p.chunk > 0))
    for tokens, top, experts, n, kb, gated in FEW_EXPERTS:
        p = plan(emu, tokens, tokens * top, experts, n, 128 * kb, gated)
        tiles.add((p.weight_tiles, gated, "values" if not p.quantize else "codes"))
        refilled.add(p.few and not p.quantize and kb > p.chunk and ("experts", kb % p.chunk > 0))
    assert tiles == {(t, g, x) for t, g in ((1, 0), (2, 0), (2, 1), (4, 1)) for x in ("values", "codes")}
    assert refilled >= {("one", True), ("experts", False)}
