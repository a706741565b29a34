"""The attention's launch plan and workspace for the 8-bit key/value cache, on the host (no GPU)."""
import ctypes

import numpy as np
import pytest

import block_quantized_weight_nq_amd as nq


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
