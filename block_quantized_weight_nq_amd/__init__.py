"""Python binding of libnq.so, the MI355X (gfx950) packed-weight decoder.

Argument marshalling only: every step of a decode runs in the library's HIP
kernels behind the C ABI of include/nq.h.  PyTorch supplies device memory
and streams.  There is no fallback: if libnq.so is missing, every call raises.

    import torch, block_quantized_weight_nq_amd as nq
    y = nq.dequantize_packed("gguf:q4_k", payload_u8_cuda, [4096, 4096], torch.bfloat16)
"""
import collections
import contextlib
import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnq.so")

NQ_OK = 0
STATUS_NAMES = {0: "NQ_OK", 1: "NQ_ERR_NULL_ARG", 2: "NQ_ERR_UNKNOWN_FORMAT", 3: "NQ_ERR_BAD_RANK",
                4: "NQ_ERR_BAD_DIM", 5: "NQ_ERR_NOT_BLOCK_ALIGNED", 6: "NQ_ERR_LENGTH_MISMATCH",
                7: "NQ_ERR_OVERFLOW", 8: "NQ_ERR_BAD_DTYPE", 9: "NQ_ERR_HIP", 10: "NQ_ERR_BAD_DIVISORS",
                11: "NQ_ERR_MISALIGNED", 12: "NQ_ERR_SCRATCH"}
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2, "f64": 3}
FAMILIES = {0: "simple", 1: "kquant", 2: "iq", 3: "fp4", 4: "ternary"}
EXPORTS = ["nq_format_count", "nq_format_by_id", "nq_format_query", "nq_validate",
           "nq_dequantize_packed", "nq_dequantize_packed_many", "nq_measure_stream", "nq_validate_nvfp4_stacked", "nq_dequantize_nvfp4_stacked",
           "nq_validate_fp8_row", "nq_dequantize_fp8_row", "nq_validate_grouped_absmax",
           "nq_quantize_grouped_absmax", "nq_validate_quantize_q8_1", "nq_quantize_q8_1",
           "nq_validate_gemv_q8_1", "nq_gemv_q8_1", "nq_validate_gemm_q8_1", "nq_gemm_q8_1_workspace", "nq_gemm_q8_1", "nq_gemm_q8_1_noalloc",
           "nq_kv_tables", "nq_kv_store", "nq_kv_load", "nq_kv_attention_workspace", "nq_kv_attention",
           "nq_quantize_fp8_block", "nq_dequantize_fp8_block", "nq_gemm_fp8_block_workspace", "nq_gemm_fp8_block",
           "nq_moe_sort_workspace", "nq_moe_sort", "nq_moe_gather", "nq_moe_combine", "nq_moe_combine_grad",
           "nq_status_string"]
GEMV_MAX_M = 8
GQ_SCHEMES = {"q4_g64_fp16": (0, 64), "q5_g64_fp16": (1, 64), "q6_g64_fp16": (2, 64), "q8_g32_fp16": (3, 32)}
KV_CODES = {"q8": 0, "e4m3": 1}
FP8_BLOCK, MOE_MAX_EXPERTS = 128, 1024
KV_DIMS, KV_BLOCKS = (64, 128, 256), (16, 32, 64, 128)
FP8_ROW_KINDS = {"fp8_e4m3fn_row_bf16": 0, "fp8_e4m3fn_row_fp16": 1}


class NqError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        msg = _lib().nq_status_string(status).decode()
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}{(' (' + what + ')') if what else ''}")


class FormatInfo(ctypes.Structure):
    _fields_ = [("id", ctypes.c_int32), ("name", ctypes.c_char_p), ("block_values", ctypes.c_int32),
                ("block_bytes", ctypes.c_int32), ("trailer_bytes", ctypes.c_int32),
                ("family", ctypes.c_int32)]

    def __repr__(self):
        return (f"FormatInfo(id={self.id}, name={self.name.decode()!r}, B={self.block_values}, "
                f"S={self.block_bytes}, trailer={self.trailer_bytes}, family={FAMILIES[self.family]})")


class TensorDesc(ctypes.Structure):
    """nq_tensor: one tensor of nq_dequantize_packed_many."""
    _fields_ = [("format", ctypes.c_int32), ("rank", ctypes.c_int32), ("shape", ctypes.POINTER(ctypes.c_int64)),
                ("payload", ctypes.c_void_p), ("nbytes", ctypes.c_uint64), ("out", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    """nq_kv_cache."""
    _fields_ = [("code", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("block", ctypes.c_int32), ("blocks", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class KvAttentionArgs(ctypes.Structure):
    """nq_kv_attention_args."""
    _fields_ = [("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("tokens", ctypes.c_int64), ("q_heads", ctypes.c_int64), ("requests", ctypes.c_int64),
                ("token_start", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_width", ctypes.c_int64), ("table_stride", ctypes.c_int64), ("window", ctypes.c_int64),
                ("max_new", ctypes.c_int64), ("max_length", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoePlanDesc(ctypes.Structure):
    """nq_moe_plan."""
    _fields_ = [("order", ctypes.c_void_p), ("places", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("top", ctypes.c_int64), ("experts", ctypes.c_int64)]


class Fp8BlockArgs(ctypes.Structure):
    """nq_fp8_block_args."""
    _fields_ = [("x", ctypes.c_void_p), ("x_row_stride", ctypes.c_int64), ("x_scales", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("weight_scales", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("gated", ctypes.c_int32), ("sorted", ctypes.c_int32)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                              "python block_quantized_weight_nq_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        c = ctypes
        L.nq_format_count.restype = c.c_int
        L.nq_format_by_id.argtypes = [c.c_int32, c.POINTER(FormatInfo)]
        L.nq_format_query.argtypes = [c.c_char_p, c.POINTER(FormatInfo)]
        L.nq_validate.argtypes = [c.c_int32, c.c_uint64, c.POINTER(c.c_int64), c.c_int32, c.c_int32,
                                  c.POINTER(c.c_uint64), c.POINTER(c.c_uint64)]
        L.nq_dequantize_packed.argtypes = [c.c_int32, c.c_void_p, c.c_uint64, c.POINTER(c.c_int64),
                                           c.c_int32, c.c_int32, c.c_void_p, c.c_void_p]
        L.nq_dequantize_packed_many.argtypes = [c.POINTER(TensorDesc), c.c_int32, c.c_int32, c.POINTER(c.c_int32),
                                                c.c_void_p]
        L.nq_measure_stream.argtypes = [c.c_void_p, c.c_uint64, c.c_void_p, c.c_uint64, c.c_int32, c.c_int32,
                                        c.c_void_p]
        L.nq_validate_nvfp4_stacked.argtypes = [c.c_uint64, c.POINTER(c.c_int64), c.c_int32, c.c_int64,
                                                c.c_int32, c.POINTER(c.c_uint64), c.POINTER(c.c_uint64)]
        L.nq_dequantize_nvfp4_stacked.argtypes = [c.c_void_p, c.c_uint64, c.POINTER(c.c_int64), c.c_int32,
                                                  c.c_int64, c.c_int32, c.c_void_p, c.c_void_p]
        L.nq_validate_fp8_row.argtypes = [c.c_int32, c.c_uint64, c.POINTER(c.c_int64), c.c_int32, c.c_int32,
                                          c.POINTER(c.c_uint64), c.POINTER(c.c_uint64)]
        L.nq_dequantize_fp8_row.argtypes = [c.c_int32, c.c_void_p, c.c_uint64, c.POINTER(c.c_int64), c.c_int32,
                                            c.c_int32, c.c_void_p, c.c_void_p]
        L.nq_validate_grouped_absmax.argtypes = [c.c_int32, c.POINTER(c.c_int64), c.c_int32, c.c_int32,
                                                 c.POINTER(c.c_uint64), c.POINTER(c.c_uint64)]
        L.nq_quantize_grouped_absmax.argtypes = [c.c_int32, c.c_void_p, c.POINTER(c.c_int64), c.c_int32, c.c_int32,
                                                 c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p]
        L.nq_validate_quantize_q8_1.argtypes = [c.POINTER(c.c_int64), c.c_int32, c.c_int32, c.POINTER(c.c_uint64)]
        L.nq_quantize_q8_1.argtypes = [c.c_void_p, c.POINTER(c.c_int64), c.c_int32, c.c_int32, c.c_void_p,
                                       c.c_void_p, c.c_void_p]
        L.nq_validate_gemv_q8_1.argtypes = [c.c_int32, c.c_uint64, c.c_int64, c.c_int64, c.c_int64]
        L.nq_gemv_q8_1.argtypes = [c.c_int32, c.c_void_p, c.c_uint64, c.c_int64, c.c_int64, c.c_void_p,
                                   c.c_int64, c.c_void_p, c.c_void_p]
        L.nq_validate_gemm_q8_1.argtypes = [c.c_int32, c.c_uint64, c.c_int64, c.c_int64, c.c_int64]
        L.nq_gemm_q8_1_workspace.argtypes = [c.c_int32, c.c_int64, c.c_int64, c.c_int64, c.POINTER(c.c_uint64)]
        L.nq_gemm_q8_1.argtypes = [c.c_int32, c.c_void_p, c.c_uint64, c.c_int64, c.c_int64, c.c_void_p,
                                   c.c_int64, c.c_void_p, c.c_void_p, c.c_uint64, c.c_void_p]
        L.nq_gemm_q8_1_noalloc.argtypes = [c.c_int32, c.c_void_p, c.c_uint64, c.c_int64, c.c_int64, c.c_void_p,
                                            c.c_int64, c.c_void_p, c.c_void_p]
        L.nq_kv_tables.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_void_p, c.c_int64, c.c_int64, c.c_void_p,
                                   c.c_int64, c.c_void_p, c.c_int32, c.c_int64, c.c_void_p, c.c_void_p, c.c_void_p,
                                   c.c_void_p, c.c_void_p, c.c_void_p]
        L.nq_kv_store.argtypes = [c.POINTER(KvCacheDesc), c.c_void_p, c.c_int64, c.c_int64, c.c_void_p, c.c_int64,
                                  c.c_int64, c.c_int64, c.c_int32, c.c_void_p, c.c_void_p, c.c_int64, c.c_void_p,
                                  c.c_void_p]
        L.nq_kv_load.argtypes = [c.POINTER(KvCacheDesc), c.c_void_p, c.c_int64, c.c_int32, c.c_void_p, c.c_void_p,
                                 c.c_void_p]
        # (the arguments: a KvAttentionArgs by reference, or its bytes)
        L.nq_kv_attention_workspace.argtypes = [c.POINTER(KvCacheDesc), c.c_void_p, c.POINTER(c.c_uint64)]
        L.nq_kv_attention.argtypes = [c.POINTER(KvCacheDesc), c.c_void_p, c.c_void_p, c.c_uint64, c.c_void_p]
        L.nq_quantize_fp8_block.argtypes = [c.c_void_p, c.c_int32, c.c_int64, c.c_int64, c.c_int64, c.c_int64, c.c_int32,
                                            c.c_void_p, c.c_void_p, c.c_void_p]
        L.nq_dequantize_fp8_block.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int64, c.c_int64, c.c_int32,
                                              c.c_int32, c.c_void_p, c.c_void_p]
        # (arguments and plans: an Fp8BlockArgs and a MoePlanDesc by reference, or their bytes)
        L.nq_gemm_fp8_block_workspace.argtypes = [c.c_void_p, c.c_void_p, c.POINTER(c.c_uint64)]
        L.nq_gemm_fp8_block.argtypes = [c.c_void_p, c.c_void_p, c.c_void_p, c.c_uint64, c.c_void_p]
        L.nq_moe_sort_workspace.argtypes = [c.c_int64, c.c_int64, c.c_int64, c.POINTER(c.c_uint64)]
        L.nq_moe_sort.argtypes = [c.c_void_p, c.c_int32, c.c_int64, c.c_int64, c.c_int64, c.c_void_p, c.c_void_p,
                                  c.c_void_p, c.c_void_p, c.c_uint64, c.c_void_p]
        L.nq_moe_gather.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int64, c.c_void_p, c.c_void_p]
        L.nq_moe_combine.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int32, c.c_int64, c.c_void_p,
                                     c.c_void_p, c.c_void_p]
        L.nq_moe_combine_grad.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_void_p, c.c_int64, c.c_int32,
                                          c.c_int64, c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p]
        L.nq_status_string.argtypes = [c.c_int]
        L.nq_status_string.restype = c.c_char_p
        _LIB = L
    return _LIB


def library():
    """The loaded ctypes library (raises if not built)."""
    return _lib()


def format_count():
    return _lib().nq_format_count()


def format_by_id(i):
    info = FormatInfo()
    st = _lib().nq_format_by_id(i, ctypes.byref(info))
    if st != NQ_OK:
        raise NqError(st, f"id {i}")
    return info


def format_query(name):
    info = FormatInfo()
    st = _lib().nq_format_query(name.encode(), ctypes.byref(info))
    if st != NQ_OK:
        raise NqError(st, repr(name))
    return info


def format_names():
    return [format_by_id(i).name.decode() for i in range(format_count())]


def _shape(shape):
    shape = [int(d) for d in shape]
    return (ctypes.c_int64 * max(1, len(shape)))(*shape), len(shape)


def _dtype_code(dtype):
    if isinstance(dtype, str):
        return DTYPE_CODES[dtype]
    import torch
    return {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float64: 3}[dtype]


def validate_status(fmt, nbytes, shape, out_dtype="f32"):
    """Raw status of nq_validate plus (elems, out_bytes)."""
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    arr, rank = _shape(shape)
    ne, nb = ctypes.c_uint64(), ctypes.c_uint64()
    code = out_dtype if isinstance(out_dtype, int) else _dtype_code(out_dtype)
    st = _lib().nq_validate(fid, nbytes, arr, rank, code, ctypes.byref(ne), ctypes.byref(nb))
    return st, ne.value, nb.value


def validate(fmt, nbytes, shape, out_dtype="f32"):
    st, ne, nb = validate_status(fmt, nbytes, shape, out_dtype)
    if st != NQ_OK:
        raise NqError(st)
    return ne, nb


def dequantize_packed_raw(fmt_id, payload_ptr, nbytes, shape, out_dtype_code, out_ptr, stream_handle):
    """Direct call of the C entry point with integer addresses; returns the status."""
    arr, rank = _shape(shape)
    return _lib().nq_dequantize_packed(fmt_id, ctypes.c_void_p(payload_ptr), nbytes, arr, rank,
                                       out_dtype_code, ctypes.c_void_p(out_ptr),
                                       ctypes.c_void_p(stream_handle))


class ManyCall:
    """A prepared nq_dequantize_packed_many call: the tensor array is built
    once and reused by every run(stream_handle) (argument marshalling only).
    descs: (format id, payload address, nbytes, shape, out address) per tensor."""

    def __init__(self, descs, out_dtype_code):
        self.n = len(descs)
        self.code = int(out_dtype_code)
        self.arr = (TensorDesc * max(1, self.n))()
        self._shapes = []
        for i, (fid, p, nbytes, shape, o) in enumerate(descs):
            sh, rank = _shape(shape)
            self._shapes.append(sh)
            self.arr[i] = TensorDesc(int(fid), rank, ctypes.cast(sh, ctypes.POINTER(ctypes.c_int64)),
                                     ctypes.c_void_p(p), int(nbytes), ctypes.c_void_p(o))
        self.failed = ctypes.c_int32(-1)

    def run_status(self, stream_handle):
        st = _lib().nq_dequantize_packed_many(self.arr if self.n else None, self.n, self.code,
                                              ctypes.byref(self.failed), ctypes.c_void_p(stream_handle))
        return st, self.failed.value

    def run(self, stream_handle):
        st, failed = self.run_status(stream_handle)
        if st != NQ_OK:
            raise NqError(st, f"tensor {failed}")


def dequantize_packed_many_raw(descs, out_dtype_code, stream_handle):
    """Direct call of nq_dequantize_packed_many.  descs: (format id, payload
    address, nbytes, shape, out address) per tensor.  Returns (status, index
    of the failing tensor or -1)."""
    return ManyCall(descs, out_dtype_code).run_status(stream_handle)


def dequantize_packed_many(items, out_dtype=None, stream=None):
    """Decode several tensors in as few launches as their formats allow.

    items: (fmt, payload, shape) or (fmt, payload, shape, out) per tensor, with
    payload a rank-1 uint8 CUDA tensor.  Returns the output tensors (new ones
    where out is not given), decoded on `stream` (default: the current stream).
    """
    import torch
    descs, outs, on = [], [], _SAME_DEVICE
    for it in items:
        fmt, payload, shape = it[0], it[1], it[2]
        out = it[3] if len(it) > 3 else None
        fid = fmt if isinstance(fmt, int) else format_query(fmt).id
        code, out, stream = _prepare(payload, shape, out_dtype if out_dtype is not None else
                                     (out.dtype if out is not None else torch.float32), out, stream)
        if not descs:
            on = _device_of(payload)
        descs.append((fid, payload.data_ptr(), payload.numel(), shape, out.data_ptr()))
        outs.append(out)
    if stream is None:
        stream = torch.cuda.current_stream()
    if out_dtype is None:
        out_dtype = outs[0].dtype if outs else torch.float32
    with on:
        st, failed = dequantize_packed_many_raw(descs, _dtype_code(out_dtype), stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"tensor {failed}")
    return outs


STREAM_NT_LOAD, STREAM_NT_STORE = 1, 2


def measure_stream_raw(src_ptr, src_bytes, dst_ptr, dst_bytes, chunks_per_thread, flags, stream_handle):
    """nq_measure_stream (measurement aid): read src_bytes, write dst_bytes; returns the status."""
    return _lib().nq_measure_stream(ctypes.c_void_p(src_ptr), int(src_bytes), ctypes.c_void_p(dst_ptr),
                                    int(dst_bytes), int(chunks_per_thread), int(flags),
                                    ctypes.c_void_p(stream_handle))


def validate_nvfp4_stacked_status(nbytes, shape, divisors, out_dtype="f32"):
    """Raw status of nq_validate_nvfp4_stacked plus (elems, out_bytes)."""
    arr, rank = _shape(shape)
    ne, nb = ctypes.c_uint64(), ctypes.c_uint64()
    code = out_dtype if isinstance(out_dtype, int) else _dtype_code(out_dtype)
    st = _lib().nq_validate_nvfp4_stacked(nbytes, arr, rank, int(divisors), code, ctypes.byref(ne),
                                          ctypes.byref(nb))
    return st, ne.value, nb.value


def dequantize_nvfp4_stacked_raw(payload_ptr, nbytes, shape, divisors, out_dtype_code, out_ptr, stream_handle):
    """Direct call of nq_dequantize_nvfp4_stacked with integer addresses; returns the status."""
    arr, rank = _shape(shape)
    return _lib().nq_dequantize_nvfp4_stacked(ctypes.c_void_p(payload_ptr), nbytes, arr, rank, int(divisors),
                                              out_dtype_code, ctypes.c_void_p(out_ptr),
                                              ctypes.c_void_p(stream_handle))


_SAME_DEVICE = contextlib.nullcontext()


def _device_of(t):
    """A context in which the CUDA tensor's device is the current one: a launch on a default stream goes to the current
    device's, and a launch plan asks that device's size."""
    import torch
    if not t.is_cuda or torch._C._cuda_getDevice() == t.get_device():
        return _SAME_DEVICE
    return torch.cuda.device(t.get_device())


def _prepare(payload, shape, out_dtype, out, stream):
    import torch
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    code = _dtype_code(out_dtype)
    if payload.dtype != torch.uint8 or payload.dim() != 1 or not payload.is_cuda:
        raise ValueError("payload must be a rank-1 torch.uint8 CUDA tensor")
    if not payload.is_contiguous():
        raise ValueError("payload must be contiguous")
    n = 1
    for d in shape:
        n *= int(d)
    if out is None:
        out = torch.empty([int(d) for d in shape], dtype=out_dtype, device=payload.device)
    elif (out.dtype != out_dtype or not out.is_contiguous() or out.numel() != n or
          (n and out.device != payload.device)):
        raise ValueError("out must be a contiguous tensor of the requested dtype, size and device")
    if stream is None:
        stream = torch.cuda.current_stream(payload.device)
    return code, out, stream


def dequantize_nvfp4_stacked(payload, shape, divisors, out_dtype=None, out=None, stream=None):
    """Decode an "nvfp4" plane stacked from `divisors` sources (one binary32
    divisor per source after the blocks) into a new (or the given) tensor."""
    code, out, stream = _prepare(payload, shape, out_dtype, out, stream)
    with _device_of(payload):
        st = dequantize_nvfp4_stacked_raw(payload.data_ptr(), payload.numel(), shape, divisors, code,
                                          out.data_ptr(), stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"nvfp4 {list(shape)} divisors={divisors}")
    return out


def validate_fp8_row_status(fmt, nbytes, shape, out_dtype="f32"):
    """Raw status of nq_validate_fp8_row plus (elems, out_bytes); fmt is the
    format name or the scale kind (0 bf16 scales, 1 fp16 scales)."""
    kind = FP8_ROW_KINDS[fmt] if isinstance(fmt, str) else int(fmt)
    arr, rank = _shape(shape)
    ne, nb = ctypes.c_uint64(), ctypes.c_uint64()
    code = out_dtype if isinstance(out_dtype, int) else _dtype_code(out_dtype)
    st = _lib().nq_validate_fp8_row(kind, nbytes, arr, rank, code, ctypes.byref(ne), ctypes.byref(nb))
    return st, ne.value, nb.value


def dequantize_fp8_row_raw(kind, payload_ptr, nbytes, shape, out_dtype_code, out_ptr, stream_handle):
    """Direct call of nq_dequantize_fp8_row with integer addresses; returns the status."""
    arr, rank = _shape(shape)
    return _lib().nq_dequantize_fp8_row(int(kind), ctypes.c_void_p(payload_ptr), nbytes, arr, rank, out_dtype_code,
                                        ctypes.c_void_p(out_ptr), ctypes.c_void_p(stream_handle))


def dequantize_fp8_row(fmt, payload, shape, out_dtype=None, out=None, stream=None):
    """Decode a row-scaled FP8 matrix ("fp8_e4m3fn_row_bf16" or "_fp16":
    N*K codes, then N scale words) into a new (or the given) [N, K] tensor."""
    code, out, stream = _prepare(payload, shape, out_dtype, out, stream)
    with _device_of(payload):
        st = dequantize_fp8_row_raw(FP8_ROW_KINDS[fmt], payload.data_ptr(), payload.numel(), shape, code,
                                    out.data_ptr(), stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"{fmt} {list(shape)}")
    return out


def validate_grouped_absmax_status(scheme, shape, in_dtype="f32"):
    """Raw status of nq_validate_grouped_absmax plus (codes bytes, scales bytes)."""
    sid = GQ_SCHEMES[scheme][0] if isinstance(scheme, str) else int(scheme)
    arr, rank = _shape(shape)
    cb, sb = ctypes.c_uint64(), ctypes.c_uint64()
    code = in_dtype if isinstance(in_dtype, int) else _dtype_code(in_dtype)
    st = _lib().nq_validate_grouped_absmax(sid, arr, rank, code, ctypes.byref(cb), ctypes.byref(sb))
    return st, cb.value, sb.value


def quantize_grouped_absmax_raw(scheme_id, x_ptr, shape, in_dtype_code, codes_ptr, scales_ptr, status_ptr,
                                stream_handle):
    """Direct call of nq_quantize_grouped_absmax with integer addresses; returns the status."""
    arr, rank = _shape(shape)
    return _lib().nq_quantize_grouped_absmax(int(scheme_id), ctypes.c_void_p(x_ptr), arr, rank, in_dtype_code,
                                             ctypes.c_void_p(codes_ptr), ctypes.c_void_p(scales_ptr),
                                             ctypes.c_void_p(status_ptr), ctypes.c_void_p(stream_handle))


def quantize_grouped_absmax(scheme, x, stream=None, check=True):
    """Encode a contiguous [N, K] CUDA tensor (float32/float16/bfloat16/float64)
    with grouped_absmax.  Returns (codes int8 [N, K], scales as int16 words
    [N, ceil(K/G)], status int32 [1]).  With check=True the call waits for
    the stream and raises NqError-like ValueError on an encoder failure."""
    import torch
    sid, G = GQ_SCHEMES[scheme]
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous rank-2 CUDA tensor")
    N, K = x.shape
    codes = torch.empty((N, K), dtype=torch.int8, device=x.device)
    scales = torch.empty((N, (K + G - 1) // G), dtype=torch.int16, device=x.device)
    status = torch.empty(1, dtype=torch.int32, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    with _device_of(x):
        st = quantize_grouped_absmax_raw(sid, x.data_ptr(), [N, K], _dtype_code(x.dtype), codes.data_ptr(),
                                         scales.data_ptr(), status.data_ptr(), stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"{scheme} {[N, K]}")
    if check:
        stream.synchronize()
        bits = int(status.item())
        if bits:
            raise ValueError(f"grouped_absmax failed: status bits {bits:#x} "
                             "(1: a source value is not finite, 2: a scale rounds past binary16)")
    return codes, scales, status


def validate_quantize_q8_1_status(shape, in_dtype="f32"):
    """Raw status of nq_validate_quantize_q8_1 plus the blocks' byte size."""
    arr, rank = _shape(shape)
    nb = ctypes.c_uint64()
    code = in_dtype if isinstance(in_dtype, int) else _dtype_code(in_dtype)
    st = _lib().nq_validate_quantize_q8_1(arr, rank, code, ctypes.byref(nb))
    return st, nb.value


def quantize_q8_1_raw(x_ptr, shape, in_dtype_code, blocks_ptr, status_ptr, stream_handle):
    """Direct call of nq_quantize_q8_1 with integer addresses; returns the status."""
    arr, rank = _shape(shape)
    return _lib().nq_quantize_q8_1(ctypes.c_void_p(x_ptr), arr, rank, in_dtype_code, ctypes.c_void_p(blocks_ptr),
                                   ctypes.c_void_p(status_ptr), ctypes.c_void_p(stream_handle))


def quantize_q8_1(x, stream=None, check=True):
    """q8_1 activation blocks of a contiguous [M, K] CUDA tensor (float32 /
    float16 / bfloat16 / float64, K % 32 == 0).  Returns (blocks uint8
    [M, K/32, 36], status int32 [1]).  With check=True the call waits for the
    stream and raises ValueError on a non-finite source or a scale past
    binary16."""
    import torch
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous rank-2 CUDA tensor")
    M, K = x.shape
    blocks = torch.empty((M, K // 32, 36), dtype=torch.uint8, device=x.device)
    status = torch.empty(1, dtype=torch.int32, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    with _device_of(x):
        st = quantize_q8_1_raw(x.data_ptr(), [M, K], _dtype_code(x.dtype), blocks.data_ptr(), status.data_ptr(),
                               stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"q8_1 {[M, K]}")
    if check:
        stream.synchronize()
        bits = int(status.item())
        if bits & 3:
            raise ValueError(f"q8_1 quantization failed: status bits {bits:#x} "
                             "(1: a source value is not finite, 2: a scale rounds past binary16)")
    return blocks, status


def validate_gemv_q8_1_status(fmt, nbytes, N, K, M):
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    return _lib().nq_validate_gemv_q8_1(fid, nbytes, N, K, M)


def gemv_q8_1_raw(fmt_id, w_ptr, nbytes, N, K, xq_ptr, M, y_ptr, stream_handle):
    """Direct call of nq_gemv_q8_1 with integer addresses; returns the status."""
    return _lib().nq_gemv_q8_1(int(fmt_id), ctypes.c_void_p(w_ptr), nbytes, N, K, ctypes.c_void_p(xq_ptr), M,
                               ctypes.c_void_p(y_ptr), ctypes.c_void_p(stream_handle))


def validate_gemm_q8_1_status(fmt, nbytes, N, K, M):
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    return _lib().nq_validate_gemm_q8_1(fid, nbytes, N, K, M)


def gemm_q8_1_workspace(fmt, N, K, M):
    """(status, workspace bytes) of the batched product for this shape on the current device."""
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    b = ctypes.c_uint64(0)
    st = _lib().nq_gemm_q8_1_workspace(fid, N, K, M, ctypes.byref(b))
    return st, b.value


def gemm_q8_1_raw(fmt_id, w_ptr, nbytes, N, K, xq_ptr, M, y_ptr, ws_ptr, ws_bytes, stream_handle):
    """Direct call of nq_gemm_q8_1 with integer addresses; returns the status."""
    return _lib().nq_gemm_q8_1(int(fmt_id), ctypes.c_void_p(w_ptr), nbytes, N, K, ctypes.c_void_p(xq_ptr), M,
                               ctypes.c_void_p(y_ptr), ctypes.c_void_p(ws_ptr), ws_bytes,
                               ctypes.c_void_p(stream_handle))


GEMM_SCRATCH_BYTES = 32 << 20


def gemm_q8_1_noalloc_raw(fmt_id, w_ptr, nbytes, N, K, xq_ptr, M, y_ptr, stream_handle):
    """nq_gemm_q8_1_noalloc (the library's static scratch as the workspace); returns the status."""
    return _lib().nq_gemm_q8_1_noalloc(fmt_id, ctypes.c_void_p(w_ptr), nbytes, N, K, ctypes.c_void_p(xq_ptr), M,
                                       ctypes.c_void_p(y_ptr), ctypes.c_void_p(stream_handle))


def _product(raw, fmt, weight, N, K, xq, out, stream):
    import torch
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    if not weight.is_cuda or not xq.is_cuda or xq.dtype != torch.uint8 or not xq.is_contiguous():
        raise ValueError("weight and xq must be CUDA uint8 tensors, xq contiguous")
    M = xq.numel() // (K // 32 * 36) if K % 32 == 0 and K > 0 else 0
    if xq.numel() != M * (K // 32) * 36:
        raise ValueError("xq holds a whole number of activation rows of K / 32 blocks")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=weight.device)
    elif out.dtype != torch.float32 or not out.is_contiguous() or out.numel() != M * N:
        raise ValueError("out must be a contiguous float32 tensor of M * N elements")
    if stream is None:
        stream = torch.cuda.current_stream(weight.device)
    with _device_of(weight):
        st = raw(fid, weight.data_ptr(), weight.numel(), N, K, xq.data_ptr(), M, out.data_ptr(), stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"{fmt} [{N}, {K}] x {M}")
    return out


def gemv_q8_1(fmt, weight, N, K, xq, out=None, stream=None):
    """y[M, N] (float32) = x[M, K] @ w[N, K]^T for a rank-1 uint8 CUDA weight
    payload of `fmt` (a "gguf:" format) and q8_1 activation blocks `xq`
    ([M, K/32, 36] uint8, as quantize_q8_1 returns), M <= 8."""
    return _product(gemv_q8_1_raw, fmt, weight, N, K, xq, out, stream)


def gemm_q8_1(fmt, weight, N, K, xq, out=None, stream=None, split=True):
    """As gemv_q8_1 for any number of activation rows M >= 1 (5 or more on
    the matrix cores).  With split=True the workspace the product may use is
    allocated from torch on `stream` (K then splits, and the weight is
    rewritten once, where the shape asks for it); split=False runs without a
    workspace."""
    import torch
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    M = xq.numel() // (K // 32 * 36) if K % 32 == 0 and K > 0 else 0
    ws, ws_bytes = None, 0
    if split and M > 0:
        with _device_of(weight):
            st, ws_bytes = gemm_q8_1_workspace(fid, N, K, M)
        if st != NQ_OK:
            raise NqError(st, f"{fmt} [{N}, {K}] x {M}")
        if ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=weight.device)
            if stream is not None:
                ws.record_stream(stream)

    def raw(fid_, w_ptr, nbytes, N_, K_, xq_ptr, M_, y_ptr, h):
        return gemm_q8_1_raw(fid_, w_ptr, nbytes, N_, K_, xq_ptr, M_, y_ptr, ws.data_ptr() if ws is not None else 0,
                             ws_bytes, h)

    return _product(raw, fmt, weight, N, K, xq, out, stream)


def dequantize_packed(fmt, payload, shape, out_dtype=None, out=None, stream=None):
    """Decode a rank-1 uint8 CUDA tensor into a new (or the given) tensor of `shape`.

    out_dtype: torch.float32 (default), torch.float16, torch.bfloat16 or torch.float64.
    The decode is enqueued on `stream` (default: the current stream).
    """
    fid = fmt if isinstance(fmt, int) else format_query(fmt).id
    code, out, stream = _prepare(payload, shape, out_dtype, out, stream)
    with _device_of(payload):
        st = dequantize_packed_raw(fid, payload.data_ptr(), payload.numel(), shape, code,
                                   out.data_ptr(), stream.cuda_stream)
    if st != NQ_OK:
        raise NqError(st, f"{fmt} {list(shape)}")
    return out


class KvCache:
    """A pool of blocks of an 8-bit key/value cache (one layer).

    k: codes [blocks, heads, block, dim], v: [blocks, heads, dim, block], both torch.int8 ("q8") or both
    torch.float8_e4m3fn ("e4m3"); k_scale, v_scale: float32 [blocks, heads].  Contiguous CUDA tensors that the
    caller owns and that the calls below update in place.  KvCache.empty() allocates a pool.
    """

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if _I32 is None:
            _torch_names()
        codes = {torch.int8: "q8", torch.float8_e4m3fn: "e4m3"}
        if k.dtype not in codes or v.dtype != k.dtype:
            raise ValueError("k and v must both be torch.int8 or both torch.float8_e4m3fn")
        if k.dim() != 4 or v.dim() != 4:
            raise ValueError("k must be [blocks, heads, block, dim] and v [blocks, heads, dim, block]")
        blocks, heads, block, dim = k.shape
        if tuple(v.shape) != (blocks, heads, dim, block):
            raise ValueError("k must be [blocks, heads, block, dim] and v [blocks, heads, dim, block]")
        if dim not in KV_DIMS or block not in KV_BLOCKS or blocks < 1 or heads < 1:
            raise ValueError(f"dim must be one of {KV_DIMS}, block one of {KV_BLOCKS}, blocks and heads at least 1")
        for s in (k_scale, v_scale):
            if s.dtype != torch.float32 or tuple(s.shape) != (blocks, heads):
                raise ValueError("scales must be float32 [blocks, heads]")
        for t in (k, v, k_scale, v_scale):
            if not t.is_cuda or t.device != k.device or not t.is_contiguous():
                raise ValueError("cache tensors must be contiguous CUDA tensors of one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.blocks, self.heads, self.block, self.dim, self.code = blocks, heads, block, dim, codes[k.dtype]
        self.device, self.index = k.device, k.get_device()
        self._workspaces = {}
        self._desc = KvCacheDesc(KV_CODES[self.code], heads, dim, block, blocks, k.data_ptr(), v.data_ptr(),
                                 k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = ctypes.byref(self._desc)

    @classmethod
    def empty(cls, blocks, heads, block, dim, code="q8", device="cuda"):
        """A pool with uninitialized contents (the calls never read what was not stored)."""
        import torch
        dtype = {"q8": torch.int8, "e4m3": torch.float8_e4m3fn}[code]
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        return cls(new((blocks, heads, block, dim), dtype), new((blocks, heads, dim, block), dtype),
                   new((blocks, heads), torch.float32), new((blocks, heads), torch.float32))


KvStep = collections.namedtuple("KvStep", "lengths token_start slots free_state status")

# A serving step makes these calls once a layer, at a few microseconds each: they compare dtypes and device indices
# in one expression (and look for the culprit only when it fails), take the raw stream, and pass
# nq_kv_attention_args as packed bytes (the fields of KvAttentionArgs, in its layout).
_ATTENTION_ARGS = struct.Struct("@PqqqqqPPPqqqqqPPif")
assert _ATTENTION_ARGS.size == ctypes.sizeof(KvAttentionArgs)
_I32 = _I64 = _F32 = _U8 = _F8 = _STREAM = _DEVICE = None
_KV_DTYPES = {}


def _torch_names():
    """torch's names that the calls below use, looked up at the first of them."""
    global _I32, _I64, _F32, _U8, _F8, _STREAM, _DEVICE
    import torch
    _KV_DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    _I64, _F32, _U8, _STREAM = torch.int64, torch.float32, torch.uint8, torch._C._cuda_getCurrentRawStream
    _DEVICE, _F8 = torch._C._cuda_getDevice, torch.float8_e4m3fn
    _I32 = torch.int32


def _on(stream, index):
    """Outputs belong to the stream that the work runs on."""
    import torch
    if stream.device.index != index:
        raise ValueError(f"stream must be one of CUDA device {index}")
    return torch.cuda.stream(stream)


def _at(index):
    """The calls' work goes to their tensors' device, whichever is the current one (as _device_of)."""
    import torch
    return torch.cuda.device(index)


def _kv_dtype(dtype):
    code = _KV_DTYPES.get(dtype)
    return _dtype_code(dtype) if code is None else code


def _refuse(index, table, requests, ints):
    """Raise for the argument that is not what the call needs: ints are (name, tensor, dtype)."""
    for name, t, dtype in ints:
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor on CUDA device {index}")
    if table is not None:
        raise ValueError(f"table must be {_I32} [{requests}, width] on CUDA device {index}, each row contiguous")


def kv_tables(lengths, added, table, ring, free_state, block, tokens, stream=None):
    """Block tables, slots and token starts of one serving step, on the GPU.

    lengths, added: int32 [requests], the tokens a request holds and its new ones (-1: it ends); table: int32
    [requests, width]; ring: int32 [ring size], the free blocks from free_state = int32 [head, count]; tokens:
    room for the step's new tokens.  table and ring are updated in place.  Returns KvStep(lengths, token_start
    [requests + 1], slots int64 [tokens], free_state, status int32 [1]); nothing changes if status is not 0 (1: too
    few free blocks, 2: a bad length, 4: more than `tokens` new tokens, 8: the ring cannot hold the blocks).
    """
    if _I32 is None:
        _torch_names()
    if not lengths.is_cuda:
        raise ValueError("lengths must be a CUDA tensor")
    index, n, i32 = lengths.get_device(), lengths.numel(), _I32
    if stream is not None:
        with _on(stream, index):
            return kv_tables(lengths, added, table, ring, free_state, block, tokens)
    if _DEVICE() != index:
        with _at(index):
            return kv_tables(lengths, added, table, ring, free_state, block, tokens)
    if not (lengths.dtype is i32 and added.dtype is i32 and ring.dtype is i32 and free_state.dtype is i32 and
            added.get_device() == index and ring.get_device() == index and free_state.get_device() == index and
            lengths.is_contiguous() and added.is_contiguous() and ring.is_contiguous() and free_state.is_contiguous() and
            table.dtype is i32 and table.get_device() == index and table.dim() == 2 and table.shape[0] == n and
            table.shape[1] > 0 and table.stride(1) == 1):
        _refuse(index, table, n, (("lengths", lengths, i32), ("added", added, i32), ("ring", ring, i32),
                                  ("free_state", free_state, i32)))
    if added.numel() != n or free_state.numel() != 2:
        raise ValueError("added must have one entry for each request and free_state two")
    words = lengths.new_empty(2 * n + 4)
    slots = lengths.new_empty(max(0, tokens), dtype=_I64)
    p = words.data_ptr()
    st = (_LIB or _lib()).nq_kv_tables(
        lengths.data_ptr(), added.data_ptr(), n, table.data_ptr(), table.shape[1], table.stride(0), ring.data_ptr(),
        ring.numel(), free_state.data_ptr(), block, tokens, p, p + 4 * n, slots.data_ptr(), p + 8 * n + 4,
        p + 8 * n + 12, _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"{n} requests, table {list(table.shape)}, block {block}, {tokens} tokens")
    new_lengths, token_start, state, status = words.split_with_sizes((n, n + 1, 2, 1))
    return KvStep(new_lengths, token_start, slots, state, status)


def _heads_of(name, x, cache, heads=None):
    shape = x.shape
    if len(shape) != 3 or shape[2] != cache.dim or (heads and shape[1] != heads) or x.get_device() != cache.index or \
            (x.stride(2) != 1 and x.numel()):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {cache.dim}] on {cache.device}, "
                         "channels contiguous")


def kv_store(cache, k, v, slots, token_start, stream=None):
    """Quantize new keys and values ([tokens, heads, dim], float32, float16 or bfloat16, any token and head strides)
    into their blocks.  slots: int64 [tokens], token_start: int32 [requests + 1] (as kv_tables returns them).
    Returns status int32 [1]: 1 a value is not finite (NaN is stored as 0, infinities saturate), 2 a slot outside
    the pool or out of order (that block's tokens are not stored)."""
    if stream is not None:
        with _on(stream, cache.index):
            return kv_store(cache, k, v, slots, token_start)
    if _DEVICE() != cache.index:
        with _at(cache.index):
            return kv_store(cache, k, v, slots, token_start)
    _heads_of("k", k, cache, cache.heads)
    _heads_of("v", v, cache, cache.heads)
    n, index = k.shape[0], cache.index
    if v.dtype is not k.dtype or v.shape[0] != n:
        raise ValueError("k and v must have one type and one number of tokens")
    if not (slots.dtype is _I64 and token_start.dtype is _I32 and slots.get_device() == index and
            token_start.get_device() == index and slots.is_contiguous() and token_start.is_contiguous()):
        _refuse(index, None, 0, (("slots", slots, _I64), ("token_start", token_start, _I32)))
    if slots.numel() < n or token_start.numel() < 2:
        raise ValueError("slots needs one entry for each token and token_start one for each request and one more")
    status = token_start.new_empty(1)
    ks, vs = k.stride(), v.stride()
    st = (_LIB or _lib()).nq_kv_store(
        cache._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], n, _kv_dtype(k.dtype), slots.data_ptr(),
        token_start.data_ptr(), token_start.numel() - 1, status.data_ptr(), _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"k {list(k.shape)} {k.dtype}")
    return status


def kv_load(cache, ids, out_dtype=None, stream=None):
    """Keys and values of whole blocks (ids: int32 [n]), each [n, block, heads, dim] in out_dtype (default float32)."""
    if stream is not None:
        with _on(stream, cache.index):
            return kv_load(cache, ids, out_dtype)
    if _DEVICE() != cache.index:
        with _at(cache.index):
            return kv_load(cache, ids, out_dtype)
    index = cache.index
    if not (ids.dtype is _I32 and ids.get_device() == index and ids.is_contiguous()):
        _refuse(index, None, 0, (("ids", ids, _I32),))
    out_dtype = out_dtype or _F32
    code = _kv_dtype(out_dtype)
    n = ids.numel()
    shape = (n, cache.block, cache.heads, cache.dim)
    k = ids.new_empty(shape, dtype=out_dtype)
    v = ids.new_empty(shape, dtype=out_dtype)
    st = (_LIB or _lib()).nq_kv_load(cache._ref, ids.data_ptr(), n, code, k.data_ptr(), v.data_ptr(), _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"{n} blocks as {out_dtype}")
    return k, v


def kv_attention(cache, q, token_start, lengths, table, scale=None, window=0, max_new=None, max_length=None,
                 return_lse=False, stream=None):
    """Causal attention of new tokens over a cache that already holds their keys and values.

    q: [tokens, q_heads, dim] (float32, float16 or bfloat16; any token and head strides), q_heads a multiple of
    cache.heads; token_start: int32 [requests + 1]; lengths: int32 [requests], new tokens included; table: int32
    [requests, width].  scale: default dim ** -0.5; window: keys a token sees at most, 0 for all.  max_new and
    max_length bound a request's new tokens and length (default: `tokens` and what the table can name); tight
    bounds save launches of idle workgroups, new tokens past max_new get 0, keys past max_length are not seen.
    Returns out in q's type and shape, and with return_lse also the natural logarithms of the sums, float32
    [tokens, q_heads].
    """
    if stream is not None:
        with _on(stream, cache.index):
            return kv_attention(cache, q, token_start, lengths, table, scale, window, max_new, max_length, return_lse)
    if _DEVICE() != cache.index:
        with _at(cache.index):
            return kv_attention(cache, q, token_start, lengths, table, scale, window, max_new, max_length, return_lse)
    _heads_of("q", q, cache)
    n, q_heads, dim = q.shape
    requests, width, index, i32 = lengths.numel(), table.shape[-1], cache.index, _I32
    if not (token_start.dtype is i32 and lengths.dtype is i32 and table.dtype is i32 and
            token_start.get_device() == index and lengths.get_device() == index and table.get_device() == index and
            token_start.is_contiguous() and lengths.is_contiguous() and table.dim() == 2 and
            table.shape[0] == requests and width > 0 and table.stride(1) == 1):
        _refuse(index, table, requests, (("token_start", token_start, i32), ("lengths", lengths, i32)))
    if token_start.numel() != requests + 1:
        raise ValueError("token_start must have one entry more than lengths")
    if max_new is None:
        max_new = max(1, n)
    if max_length is None:
        max_length = width * cache.block
    if scale is None:
        scale = dim ** -0.5
    code = _kv_dtype(q.dtype)
    lib, ref, strides = _LIB or _lib(), cache._ref, q.stride()
    out = q.new_empty((n, q_heads, dim))
    lse = q.new_empty((n, q_heads), dtype=_F32) if return_lse else None
    args = _ATTENTION_ARGS.pack(q.data_ptr(), strides[0], strides[1], n, q_heads, requests, token_start.data_ptr(),
                                lengths.data_ptr(), table.data_ptr(), width, table.stride(0), window, max_new,
                                max_length, out.data_ptr(), lse.data_ptr() if return_lse else 0, code, scale)
    # the workspace is a function of the sizes alone: asked for once for each
    sizes = (n, q_heads, requests, width, window, max_new, max_length, code)
    need = cache._workspaces.get(sizes)
    st = NQ_OK
    if need is None:
        asked = ctypes.c_uint64()
        st = lib.nq_kv_attention_workspace(ref, args, asked)
        need = asked.value
        if st == NQ_OK:
            if len(cache._workspaces) >= 1024:
                cache._workspaces.clear()
            cache._workspaces[sizes] = need
    if st == NQ_OK:
        ws = q.new_empty(need, dtype=_U8) if need else None
        st = lib.nq_kv_attention(ref, args, ws.data_ptr() if need else None, need, _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"q {list(q.shape)} {q.dtype}, {requests} requests, table {list(table.shape)}, "
                          f"window {window}, max_new {max_new}, max_length {max_length}")
    return (out, lse) if return_lse else out


# --- E4M3 blocks of 128, and rows sorted by expert ----------------------------------------------------------------

# No call records an autograd graph: results do not require gradients, whatever their inputs do.  moe_combine_grad and
# moe_combine (for moe_gather) give the gradients that there are; a torch.autograd.Function around them is the caller's.
# Types go to the library as _KV_DTYPES' codes, -1 for what it refuses as NQ_ERR_BAD_DTYPE.
_BLOCK_ARGS, _PLAN_ARGS = struct.Struct("@PqPPPPqqqiiii"), struct.Struct("@PPPqqq")
assert _BLOCK_ARGS.size == ctypes.sizeof(Fp8BlockArgs) and _PLAN_ARGS.size == ctypes.sizeof(MoePlanDesc)
_SORT_WORKSPACES = {}


def _block_shapes(shape, tile):
    """(matrices, rows, cols, shape of the scales) of a [rows, cols] or [matrices, rows, cols] tensor."""
    if tile not in (1, FP8_BLOCK):
        raise ValueError(f"tile must be 1 or {FP8_BLOCK}")
    if len(shape) not in (2, 3):
        raise ValueError("a matrix [rows, cols] or several [matrices, rows, cols] are wanted")
    rows, cols = shape[-2], shape[-1]
    return (shape[0] if len(shape) == 3 else 1), rows, cols, (*shape[:-2], -(-rows // tile), cols // FP8_BLOCK)


def quantize_fp8_block(x, tile=1, stream=None):
    """E4M3 codes and binary32 scales of x, [rows, cols] or [matrices, rows, cols] (float32, float16 or bfloat16,
    columns contiguous, any row stride): one scale for each 128 columns of `tile` rows, 1 for activations and 128 for
    weights.  cols must be a multiple of 128.  What is not finite becomes NaN.  Returns (codes float8_e4m3fn in x's
    shape, scales float32 [..., ceil(rows / tile), cols / 128])."""
    if _I32 is None:
        _torch_names()
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    index = x.get_device()
    if stream is not None:
        with _on(stream, index):
            return quantize_fp8_block(x, tile)
    if _DEVICE() != index:
        with _at(index):
            return quantize_fp8_block(x, tile)
    shape, strides = x.shape, x.stride()
    if tile == 1 and len(shape) == 2:  # (activations: a call in every layer)
        matrices, (rows, cols) = 1, shape
        scales_shape = (rows, cols // FP8_BLOCK)
    else:
        matrices, rows, cols, scales_shape = _block_shapes(shape, tile)
    if strides[-1] != 1 and x.numel() or (matrices > 1 and strides[0] != rows * strides[1]):
        raise ValueError("x must have contiguous columns, and matrices must follow each other row by row")
    codes = x.new_empty(shape, dtype=_F8)
    scales = x.new_empty(scales_shape, dtype=_F32)
    st = (_LIB or _lib()).nq_quantize_fp8_block(x.data_ptr(), _KV_DTYPES.get(x.dtype, -1), matrices, rows, cols, strides[-2],
                                                tile, codes.data_ptr(), scales.data_ptr(), _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"x {list(shape)} {x.dtype}, tile {tile}")
    return codes, scales


def _scales_of(name, scales, shape, index):
    if scales.dtype is not _F32 or tuple(scales.shape) != tuple(shape) or scales.get_device() != index or \
            not scales.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor {list(shape)} on CUDA device {index}")


def dequantize_fp8_block(codes, scales, tile=1, out_dtype=None, stream=None):
    """The values of E4M3 codes and their scales (as quantize_fp8_block returns them) in out_dtype (default float32)."""
    if _I32 is None:
        _torch_names()
    if not codes.is_cuda or codes.dtype is not _F8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous float8_e4m3fn CUDA tensor")
    index = codes.get_device()
    if stream is not None:
        with _on(stream, index):
            return dequantize_fp8_block(codes, scales, tile, out_dtype)
    if _DEVICE() != index:
        with _at(index):
            return dequantize_fp8_block(codes, scales, tile, out_dtype)
    shape = codes.shape
    matrices, rows, cols, scales_shape = _block_shapes(shape, tile)
    if scales.dtype is not _F32 or scales.shape != scales_shape or scales.get_device() != index or not scales.is_contiguous():
        _scales_of("scales", scales, scales_shape, index)
    out_dtype = out_dtype or _F32
    out = codes.new_empty(shape, dtype=out_dtype)
    st = (_LIB or _lib()).nq_dequantize_fp8_block(codes.data_ptr(), scales.data_ptr(), matrices, rows, cols, tile,
                                                  _KV_DTYPES.get(out_dtype, -1), out.data_ptr(), _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"codes {list(codes.shape)} as {out.dtype}")
    return out


class Fp8Weight:
    """A linear layer's weight in E4M3 blocks: codes float8_e4m3fn [N, K], or [experts, N, K] for one of each expert;
    scales float32 [..., ceil(N / 128), K / 128].  Contiguous CUDA tensors that the caller owns."""

    def __init__(self, codes, scales):
        if _I32 is None:
            _torch_names()
        if codes.dtype is not _F8 or codes.dim() not in (2, 3) or not codes.is_cuda or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous float8_e4m3fn CUDA tensor [N, K] or [experts, N, K]")
        self.N, self.K = codes.shape[-2:]
        self.experts = codes.shape[0] if codes.dim() == 3 else 0
        if self.N < 1 or self.K < 1 or self.K % FP8_BLOCK or (codes.dim() == 3 and not 1 <= self.experts <= MOE_MAX_EXPERTS):
            raise ValueError(f"N and K must be positive, K a multiple of {FP8_BLOCK}, experts 1 to {MOE_MAX_EXPERTS}")
        self.device, self.index = codes.device, codes.get_device()
        _scales_of("scales", scales, (*codes.shape[:-2], -(-self.N // FP8_BLOCK), self.K // FP8_BLOCK), self.index)
        self.codes, self.scales = codes, scales
        self._workspaces = {}

    @classmethod
    def quantize(cls, weight, stream=None):
        """From values: [N, K] or [experts, N, K] (float32, float16 or bfloat16)."""
        return cls(*quantize_fp8_block(weight, FP8_BLOCK, stream))


class MoePlan:
    """A router's pairs (token, choice) in the experts' order, as moe_sort returns them: order int32 [tokens * top], the
    pair token * top + choice at each place (-1 behind the last), places int32 [tokens, top], the place of each pair
    (-1: left out), offsets int32 [experts + 1], the first place of each expert."""

    def __init__(self, order, places, offsets):
        if _I32 is None:
            _torch_names()
        if not order.is_cuda:
            raise ValueError("the plan's tensors must be CUDA tensors")
        self.index = order.get_device()
        _refuse_other(self.index, (("order", order, _I32), ("places", places, _I32), ("offsets", offsets, _I32)))
        if places.dim() != 2 or order.numel() != places.numel() or not 2 <= offsets.numel() <= MOE_MAX_EXPERTS + 1:
            raise ValueError("places must be [tokens, top], order one entry for each pair, offsets experts + 1")
        tokens, top = places.shape
        self._take(order, places, offsets, order.data_ptr(), places.data_ptr(), offsets.data_ptr(), tokens, top,
                   offsets.numel() - 1)

    def _take(self, order, places, offsets, order_at, places_at, offsets_at, tokens, top, experts):
        self.order, self.places, self.offsets = order, places, offsets
        self.tokens, self.top, self.pairs, self.experts = tokens, top, tokens * top, experts
        self._ref = _PLAN_ARGS.pack(order_at, places_at, offsets_at, tokens, top, experts)

    def __reduce__(self):  # (a copy has addresses of its own)
        return MoePlan, (self.order, self.places, self.offsets)

    @property
    def device(self):
        return self.order.device


def _refuse_other(index, ints):
    """As _refuse, where any of them is not what the call needs."""
    for _, t, dtype in ints:
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            _refuse(index, None, 0, ints)


def _rows_of(name, x, rows, cols, index):
    shape = x.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols) or \
            x.get_device() != index or (x.stride(1) != 1 and x.numel()):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'cols' if cols is None else cols}] on CUDA "
                         f"device {index}, columns contiguous")


def _block_product(weight, x, x_scales, plan, sorted_rows, gated, out_dtype):
    index, n, k = weight.index, weight.N, weight.K
    if plan is None:
        rows, wanted = x.shape[0], None
        out_rows = rows
    else:
        if plan.index != index or plan.experts != weight.experts:
            raise ValueError("the plan must be one of the weight's experts and device")
        wanted = rows = plan.pairs if sorted_rows else plan.tokens
        out_rows = plan.pairs
    _rows_of("x", x, wanted, k, index)
    pointer, stride, dtype = x.data_ptr(), x.stride(0), x.dtype
    if x_scales is None:
        code, xs = _KV_DTYPES.get(dtype, -1), 0
        out_dtype = out_dtype or dtype
    else:
        if dtype is not _F8:
            raise ValueError("x must be float8_e4m3fn where x_scales is given")
        _scales_of("x_scales", x_scales, (rows, k // FP8_BLOCK), index)
        code, xs = 3, x_scales.data_ptr()
        out_dtype = out_dtype or _F32
    out_code = _KV_DTYPES.get(out_dtype, -1)
    out = x.new_empty((out_rows, n // 2 if gated else n), dtype=out_dtype)
    lib, ref = _LIB or _lib(), plan._ref if plan is not None else None
    args = _BLOCK_ARGS.pack(pointer, stride, xs, weight.codes.data_ptr(), weight.scales.data_ptr(), out.data_ptr(), rows, n, k,
                            code, out_code, gated, sorted_rows)
    # the workspace is a function of these alone: asked for once for each
    sizes = (rows, out_rows, code, out_code, gated, stride, pointer & 15, sorted_rows)
    need = weight._workspaces.get(sizes)
    st = NQ_OK
    if need is None:
        asked = ctypes.c_uint64()
        st = lib.nq_gemm_fp8_block_workspace(args, ref, asked)
        need = asked.value
        if st == NQ_OK:
            if len(weight._workspaces) >= 1024:
                weight._workspaces.clear()
            weight._workspaces[sizes] = need
    if st == NQ_OK:
        ws = x.new_empty(need, dtype=_U8) if need else None
        st = lib.nq_gemm_fp8_block(args, ref, ws.data_ptr() if need else None, need, _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"x {list(x.shape)} {dtype}, weight {list(weight.codes.shape)}, gated {gated}, out {out_dtype}")
    return out


def gemm_fp8_block(weight, x, x_scales=None, gated=False, out_dtype=None, stream=None):
    """x @ w^T for an Fp8Weight [N, K].

    x: [rows, K] float32, float16 or bfloat16 (any row stride), rounded to E4M3 blocks of one row and 128 columns within
    the call; or codes float8_e4m3fn with x_scales float32 [rows, K / 128], as quantize_fp8_block returns them.
    gated: the weight's first N / 2 rows are gates, the others up (N a multiple of 256); returns silu(gate) * up,
    [rows, N / 2].  out_dtype: default x's type (float32 for codes).  float32 outputs and calls of up to 16 rows have
    exact products and binary32 sums; 16-bit outputs of more rows use the 8-bit matrix instructions, which drop up to
    2^-10 of the largest of each eight products: less than the output's rounding, unless products cancel.  Ask for
    float32 where that matters (include/nq.h states the arithmetic).  No autograd graph is recorded, and the product has no
    gradient.
    """
    if weight.experts:
        raise ValueError("an [experts, N, K] weight takes moe_gemm_fp8_block")
    if stream is not None:
        with _on(stream, weight.index):
            return _block_product(weight, x, x_scales, None, False, bool(gated), out_dtype)
    if _DEVICE() != weight.index:
        with _at(weight.index):
            return _block_product(weight, x, x_scales, None, False, bool(gated), out_dtype)
    return _block_product(weight, x, x_scales, None, False, bool(gated), out_dtype)


def moe_gemm_fp8_block(weight, x, plan, x_scales=None, sorted_rows=False, gated=False, out_dtype=None, stream=None):
    """Each expert's product with its own rows, in the plan's order: [pairs, N] (gated: [pairs, N / 2]), zeros behind the
    last place.  weight: Fp8Weight [experts, N, K]; x: one row for each token, which the product takes in the plan's
    order, or with sorted_rows one for each place (as a product before this one returned them).  The other arguments
    are gemm_fp8_block's; "up to 16 rows" is tokens * top / experts.  No autograd graph is recorded."""
    if not weight.experts:
        raise ValueError("an [N, K] weight takes gemm_fp8_block")
    if stream is not None:
        with _on(stream, weight.index):
            return _block_product(weight, x, x_scales, plan, bool(sorted_rows), bool(gated), out_dtype)
    if _DEVICE() != weight.index:
        with _at(weight.index):
            return _block_product(weight, x, x_scales, plan, bool(sorted_rows), bool(gated), out_dtype)
    return _block_product(weight, x, x_scales, plan, bool(sorted_rows), bool(gated), out_dtype)


def moe_sort(ids, experts, stream=None):
    """The pairs of a router's choices, ids [tokens, top] (int32 or int64), sorted by expert; those outside 0 ..
    experts - 1 are left out.  Returns a MoePlan; nothing is copied to the host."""
    if _I32 is None:
        _torch_names()
    if not ids.is_cuda or ids.dim() != 2 or ids.dtype not in (_I32, _I64) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA tensor [tokens, top] of int32 or int64")
    index = ids.get_device()
    if stream is not None:
        with _on(stream, index):
            return moe_sort(ids, experts)
    if _DEVICE() != index:
        with _at(index):
            return moe_sort(ids, experts)
    tokens, top = ids.shape
    if not 1 <= experts <= MOE_MAX_EXPERTS or top < 1:
        raise ValueError(f"experts must be 1 to {MOE_MAX_EXPERTS} and top at least 1")
    pairs, lib = tokens * top, _LIB or _lib()
    need, st = _SORT_WORKSPACES.get((pairs, experts)), NQ_OK  # a function of these alone: asked for once for each
    if need is None:
        asked = ctypes.c_uint64()
        st = lib.nq_moe_sort_workspace(tokens, top, experts, asked)
        need = asked.value
        if st == NQ_OK:
            if len(_SORT_WORKSPACES) >= 1024:
                _SORT_WORKSPACES.clear()
            _SORT_WORKSPACES[pairs, experts] = need
    if st == NQ_OK:
        # one allocation: order, places, offsets, workspace
        words = ids.new_empty(2 * pairs + experts + 1 + need // 4, dtype=_I32)
        order_at = words.data_ptr()
        places_at = order_at + 4 * pairs
        offsets_at = places_at + 4 * pairs
        st = lib.nq_moe_sort(ids.data_ptr(), ids.dtype is _I64, tokens, top, experts, order_at, places_at, offsets_at,
                             offsets_at + 4 * (experts + 1) if need else None, need, _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"ids {list(ids.shape)}, {experts} experts")
    parts = words.split_with_sizes((pairs, pairs, experts + 1, need // 4) if need else (pairs, pairs, experts + 1))
    plan = MoePlan.__new__(MoePlan)
    plan.index = index
    plan._take(parts[0], parts[1].view(tokens, top), parts[2], order_at, places_at, offsets_at, tokens, top, experts)
    return plan


def moe_gather(x, plan, stream=None):
    """The rows of x [tokens, cols] (any type, columns contiguous) in the plan's order, [pairs, cols], zeros behind the last
    place.  No autograd graph is recorded: the gradient of x is moe_combine(gradient of the rows, plan)."""
    index = plan.index
    if stream is not None:
        with _on(stream, index):
            return moe_gather(x, plan)
    if _DEVICE() != index:
        with _at(index):
            return moe_gather(x, plan)
    shape, strides = x.shape, x.stride()
    if len(shape) != 2 or shape[0] != plan.tokens or x.get_device() != index or strides[1] != 1:
        _rows_of("x", x, plan.tokens, None, index)
    size, cols = x.element_size(), shape[1]
    out = x.new_empty((plan.pairs, cols))
    st = (_LIB or _lib()).nq_moe_gather(plan._ref, x.data_ptr(), cols * size, strides[0] * size, out.data_ptr(), _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"x {list(x.shape)} {x.dtype}")
    return out


def _weights_of(weights, plan):
    if weights.dtype is not _F32 or weights.shape != plan.places.shape or weights.get_device() != plan.index or \
            not weights.is_contiguous():
        _scales_of("weights", weights, (plan.tokens, plan.top), plan.index)
    return weights.data_ptr()


def moe_combine(rows, plan, weights=None, stream=None):
    """The sorted rows [pairs, cols] (float32, float16 or bfloat16) back to their tokens: [tokens, cols], each the sum of
    its rows times weights (float32 [tokens, top], 1 if not given), summed in binary32 in the order of the choices.  No
    autograd graph is recorded: moe_combine_grad gives the gradients."""
    index = plan.index
    if stream is not None:
        with _on(stream, index):
            return moe_combine(rows, plan, weights)
    if _DEVICE() != index:
        with _at(index):
            return moe_combine(rows, plan, weights)
    shape, strides, tokens = rows.shape, rows.stride(), plan.tokens
    if len(shape) != 2 or shape[0] != plan.pairs or rows.get_device() != index or strides[1] != 1:
        _rows_of("rows", rows, plan.pairs, None, index)
    cols = shape[1]
    out = rows.new_empty((tokens, cols))
    st = (_LIB or _lib()).nq_moe_combine(plan._ref, rows.data_ptr(), strides[0], _KV_DTYPES.get(rows.dtype, -1), cols,
                                         None if weights is None else _weights_of(weights, plan), out.data_ptr(),
                                         _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"rows {list(rows.shape)} {rows.dtype}")
    return out


def moe_combine_grad(grad, rows, plan, weights=None, stream=None):
    """The gradients of moe_combine(rows, plan, weights) for its result's gradient grad [tokens, cols] (rows' type):
    (grad_rows [pairs, cols] in that type, 0 behind the last place; grad_weights float32 [tokens, top], 0 for pairs left
    out, None without weights).  For a torch.autograd.Function of the caller's, since moe_combine records no graph."""
    index = plan.index
    if stream is not None:
        with _on(stream, index):
            return moe_combine_grad(grad, rows, plan, weights)
    if _DEVICE() != index:
        with _at(index):
            return moe_combine_grad(grad, rows, plan, weights)
    pairs, shape, strides, grad_shape, grad_strides = plan.pairs, rows.shape, rows.stride(), grad.shape, grad.stride()
    if len(shape) != 2 or shape[0] != pairs or rows.get_device() != index or strides[1] != 1:
        _rows_of("rows", rows, pairs, None, index)
    cols, dtype = shape[1], rows.dtype
    if len(grad_shape) != 2 or grad_shape[0] != plan.tokens or grad_shape[1] != cols or grad.get_device() != index or \
            grad_strides[1] != 1:
        _rows_of("grad", grad, plan.tokens, cols, index)
    if grad.dtype is not dtype:
        raise ValueError("grad must have the rows' type")
    out = rows.new_empty((pairs, cols))
    pointer = out_weights = out_pointer = None
    if weights is not None:
        pointer = _weights_of(weights, plan)
        out_weights = weights.new_empty((plan.tokens, plan.top))
        out_pointer = out_weights.data_ptr()
    st = (_LIB or _lib()).nq_moe_combine_grad(plan._ref, grad.data_ptr(), grad_strides[0], rows.data_ptr(), strides[0],
                                              _KV_DTYPES.get(dtype, -1), cols, pointer, out.data_ptr(), out_pointer,
                                              _STREAM(index))
    if st != NQ_OK:
        raise NqError(st, f"rows {list(rows.shape)} {rows.dtype}")
    return out, out_weights
