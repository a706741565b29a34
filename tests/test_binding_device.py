"""The binding's calls run on their tensors' device, whichever is the current one (no GPU: stand-ins for the tensors,
the device calls and the library)."""
import types

import pytest
import torch

import block_quantized_weight_nq_amd as nq


class Tensor:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096

    def stride(self, i=None):
        s = [self.shape[j + 1:].numel() for j in range(len(self.shape))]
        return tuple(s) if i is None else s[i]

    def new_empty(self, shape, dtype=None):
        return Tensor([shape] if isinstance(shape, int) else shape, dtype or self.dtype, self.index)

    def split_with_sizes(self, sizes):
        return [Tensor([n], self.dtype, self.index) for n in sizes]


class Library:
    """Notes the device that is current at each launch."""

    def __init__(self, state):
        self.state = state

    def __getattr__(self, name):
        def call(*args):
            self.state.calls.append((name, self.state.device))
            return 0
        return call


@pytest.fixture
def gpus(monkeypatch):
    state = types.SimpleNamespace(device=0, calls=[], streams=[])

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state.device = state.device, self.index

        def __exit__(self, *a):
            state.device = self.before

    class Stream:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, state.device = state.device, self.stream.device.index
            state.streams.append(self.stream)

        def __exit__(self, *a):
            state.device = self.before

    def raw_stream(index):
        return 0

    nq._torch_names()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.device, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(
        [shape] if isinstance(shape, int) else shape, dtype, device.index))
    monkeypatch.setattr(nq, "_DEVICE", lambda: state.device, raising=False)
    monkeypatch.setattr(nq, "_STREAM", raw_stream)
    monkeypatch.setattr(nq, "format_query", lambda fmt: types.SimpleNamespace(id=0))
    monkeypatch.setattr(nq, "_LIB", Library(state))
    return state


def kv_calls(index):
    i32 = lambda *shape: Tensor(shape, torch.int32, index)  # noqa: E731
    cache = nq.KvCache(Tensor((4, 2, 16, 64), torch.int8, index), Tensor((4, 2, 64, 16), torch.int8, index),
                       Tensor((4, 2), torch.float32, index), Tensor((4, 2), torch.float32, index))
    x = Tensor((3, 2, 64), torch.float16, index)
    return [
        lambda **kw: nq.kv_tables(i32(2), i32(2), i32(2, 5), i32(4), i32(2), 16, 3, **kw),
        lambda **kw: nq.kv_store(cache, x, x, Tensor((3,), torch.int64, index), i32(3), **kw),
        lambda **kw: nq.kv_load(cache, i32(2), **kw),
        lambda **kw: nq.kv_attention(cache, Tensor((3, 4, 64), torch.float16, index), i32(3), i32(2), i32(2, 5), **kw)]


def weight_calls(index):
    u8 = lambda *shape: Tensor(shape, torch.uint8, index)  # noqa: E731
    x = Tensor((2, 64), torch.float32, index)
    return [
        lambda: nq.dequantize_packed("gguf:q4_0", u8(36), [2, 32]),
        lambda: nq.dequantize_packed_many([("gguf:q4_0", u8(18), [1, 32]), ("gguf:q4_0", u8(18), [1, 32])]),
        lambda: nq.dequantize_nvfp4_stacked(u8(40), [2, 32], 1),
        lambda: nq.dequantize_fp8_row("fp8_e4m3fn_row_bf16", u8(68), [2, 32]),
        lambda: nq.quantize_grouped_absmax("q8_g32_fp16", x, check=False),
        lambda: nq.quantize_q8_1(x, check=False),
        lambda: nq.gemv_q8_1("gguf:q4_0", u8(36), 2, 32, u8(1, 1, 36)),
        lambda: nq.gemm_q8_1("gguf:q4_0", u8(36), 2, 32, u8(9, 1, 36))]


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("calls", [kv_calls, weight_calls])
def test_calls_run_on_their_tensors_device(gpus, calls, index):
    for call in calls(index):
        gpus.calls.clear()
        call()
        assert gpus.calls and all(device == index for _, device in gpus.calls), gpus.calls
        assert gpus.device == 0


def test_a_stream_is_of_the_tensors_device(gpus):
    for call in kv_calls(1):
        gpus.calls.clear()
        call(stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
        assert gpus.calls and all(device == 1 for _, device in gpus.calls)
        gpus.calls.clear()
        with pytest.raises(ValueError, match="stream"):
            call(stream=types.SimpleNamespace(device=torch.device("cuda", 0)))
        assert not gpus.calls and gpus.device == 0
