"""CPU checks of the serving binding and entry points beside tests/test_serving_refusals.py."""
import ctypes

import pytest
import torch

from quantized_attention_block_b200 import build as libbuild
from quantized_attention_block_b200 import sage

P16 = 1 << 20  # an aligned address that no call below reaches
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return sage.lib()


@pytest.mark.parametrize("zero_tail", [4, -1, 8])
def test_window_zero_tail_is_two_bits(L, zero_tail):
    p = sage.SageWindowParams(1, 4, 2, 100, 64, 0, 0, 16, 0, 0.0, zero_tail)
    assert L.sage_attn_window_fwd(P16, P16, P16, P16, None, P16, ctypes.byref(p), None) == 1


def test_evict_counts_its_rows(L):
    """Sequences times heads is the kernels' grid: below 2^31."""
    c = sage.SageKvCache(65535, 64, 0, 0, 16, 8, 0, P16, P16, None, None, P16)
    s = sage.SageKvSeqs(65535, 4, P16, P16)
    assert L.sage_kv_evict(ctypes.byref(c), ctypes.byref(s), P16 + 64, 2, 32, 4, 8, P16 + 64, P16, None) == 1


def workspace(L, max_pages, window=0, sinks=0, B=2, Hq=4, weight=None, page=16):
    c = sage.SageKvCache(2, 64, 0, 0, page, 8, 0, P16, P16, None, None, weight)
    s = sage.SageKvSeqs(B, max_pages, P16, P16)
    p = sage.SageDecodeParams(Hq, window, sinks, 0.0)
    return L.sage_decode_workspace_bytes(ctypes.byref(c), ctypes.byref(s), ctypes.byref(p))


def test_decode_workspace_sizes(L):
    """Nothing to join up to 32 blocks of 16 keys (or a window that sees no more), or up to 128 with 296 rows."""
    assert workspace(L, 32) == 256 and workspace(L, 33) > 256
    assert workspace(L, 1000, window=400, sinks=4) == 256 and workspace(L, 1000, window=512) > 256
    assert workspace(L, 128, B=148) == 256 and workspace(L, 129, B=148) > 256 and workspace(L, 128, B=147) > 256
    # more than 16 heads of a group are several rows of work
    assert workspace(L, 128, B=50, Hq=2 * 48) == 256
    # the weights' scores: a float for each query head and slot that a call can see
    assert workspace(L, 32, weight=P16) >= 4 * 2 * 4 * 512
    assert workspace(L, 1000, weight=P16, window=64, sinks=1) < workspace(L, 1000, weight=P16)


def test_expect_says_what_is_wrong():
    t = torch.zeros((2, 3), dtype=torch.int32)
    sage._expect("t", t, (2, 3), torch.int32)
    for shape, dtype, x, words in (((2, 4), torch.int32, t, "shape"), ((2, None), torch.int64, t, "int64"),
                                   ((3, 2), torch.int32, t.T, "contiguous"), ((1,), torch.int32, 5, "tensor")):
        with pytest.raises(ValueError, match=words):
            sage._expect("t", x, shape, dtype)


def test_calls_want_one_cuda_device():
    c = sage.KVCache.alloc(8, 16, 2, 64, device="cpu")
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((2, 4, 64), dtype=BF)
    for call in (lambda: sage.sage_attn_decode(q, c, table, lens), lambda: sage.sage_attn_decode(q.to("meta"), c, table, lens),
                 lambda: sage.sage_kv_append(q[:, :2, None], q[:, :2, None], c, table, lens)):
        with pytest.raises(ValueError, match="device|contiguous"):
            call()
    for bad in (dict(window=-1), dict(sinks=2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            sage.sage_attn_decode(q, c, table, lens, **bad)
