"""Tensors inside larger buffers whose other bytes are known, for calls of the C ABI: what a call writes outside of an output
changes them, what it reads outside of an input shows in its results."""
import torch

BAND = 1 << 20  # bytes on each side
MARK = 0xA5     # of outputs and workspaces
POISON = 0xFF   # of inputs: NaN as binary32, binary16, bfloat16 and E4M3


class Guarded:
    def __init__(self, shape, dtype, data=None, around=MARK):
        """A tensor of zeros, or of `data`, between two bands of the byte `around`."""
        size = torch.empty((), dtype=dtype).element_size()
        n = size
        for s in shape:
            n *= s
        self.n, self.around = n, around
        self.buffer = torch.full((2 * BAND + n,), around, dtype=torch.uint8, device="cuda:0")
        self.inside = self.buffer[BAND:BAND + n]
        self.inside.zero_()
        self.tensor = self.inside.view(dtype).view(shape)
        if data is not None:
            self.tensor.copy_(torch.as_tensor(data))
        self.before = self.inside.clone() if data is not None else None
        self.ptr = self.buffer.data_ptr() + BAND

    def check(self, what):
        bands = torch.cat([self.buffer[:BAND], self.buffer[BAND + self.n:]])
        changed = torch.nonzero(bands != self.around).flatten()
        assert changed.numel() == 0, f"{what}: {changed.numel()} bytes outside were written, the first at {int(changed[0]) - BAND}"
        if self.before is not None:
            assert torch.equal(self.inside, self.before), f"{what}: an input was written"


def given(data, dtype):
    """An input."""
    data = torch.as_tensor(data)
    if dtype is torch.float8_e4m3fn:
        g = Guarded(data.shape, torch.uint8, data, POISON)
        g.tensor = g.tensor.view(dtype)
        return g
    return Guarded(data.shape, dtype, data, POISON)
