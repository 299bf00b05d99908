"""CPU checks of the serving entry points: argument errors of the C functions
(returned on the host, before any CUDA call) and of the Python binding."""
import ctypes

import pytest
import torch

from quantized_attention_block_b200 import build as libbuild
from quantized_attention_block_b200 import sage

P16 = 1 << 20  # an aligned address that no call below reaches


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return sage.lib()


def cache(**kw):
    base = dict(Hkv=2, d=64, dtype=0, quantized=0, page_size=16, n_pages=8, layout=0, k_pages=P16, v_pages=P16,
                k_scale=None, v_scale=None, weight=None)
    base.update(kw)
    return sage.SageKvCache(**base)


def seqs(**kw):
    base = dict(B=2, max_pages=4, table=P16, lens=P16)
    base.update(kw)
    return sage.SageKvSeqs(**base)


def decode(L, c, s, Hq=4, window=0, sinks=0, sm_scale=0.0, q=P16, o=P16, km=None, ws=P16, ws_bytes=1 << 30):
    p = sage.SageDecodeParams(Hq, window, sinks, sm_scale)
    return L.sage_attn_decode(q, o, None, km, ctypes.byref(c), ctypes.byref(s), ctypes.byref(p), ws, ws_bytes, None)


BAD_CACHE = [(dict(d=96), 2), (dict(dtype=2), 3), (dict(page_size=8), 1), (dict(page_size=48), 1),
             (dict(page_size=2048), 1), (dict(n_pages=0), 1), (dict(Hkv=0), 1), (dict(layout=2), 1),
             (dict(quantized=2), 1), (dict(k_pages=None), 1), (dict(v_pages=P16 + 2), 8), (dict(quantized=1), 1),
             (dict(quantized=1, k_scale=P16, v_scale=P16 + 4), 8), (dict(weight=P16 + 1), 8)]
BAD_SEQS = [(dict(B=0), 1), (dict(B=70000), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 26), 1),
            (dict(table=None), 1), (dict(lens=None), 1), (dict(lens=P16 + 2), 8)]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches_are_refused(L, kw, want):
    c, s = cache(**kw), seqs()
    assert decode(L, c, s) == want
    assert L.sage_kv_append(P16, P16, None, None, 1, 0, ctypes.byref(c), ctypes.byref(s), None) == want
    c.weight = c.weight or P16
    assert L.sage_kv_evict(ctypes.byref(c), ctypes.byref(s), P16 + 64, 4, 16, 0, 0, P16 + 64, P16, None) == want


@pytest.mark.parametrize("kw,want", BAD_SEQS)
def test_bad_sequences_are_refused(L, kw, want):
    c, s = cache(weight=P16), seqs(**kw)
    assert decode(L, c, s) == want
    assert L.sage_kv_append(P16, P16, None, None, 1, 0, ctypes.byref(c), ctypes.byref(s), None) == want
    assert L.sage_kv_evict(ctypes.byref(c), ctypes.byref(s), P16 + 64, 4, 16, 0, 0, P16 + 64, P16, None) == want


def test_decode_arguments(L):
    c, s = cache(), seqs()
    nan, inf = float("nan"), float("inf")
    for kw in (dict(Hq=0), dict(Hq=3), dict(window=-1), dict(sinks=-1), dict(sm_scale=nan), dict(sm_scale=inf),
               dict(q=None), dict(o=None), dict(ws=None), dict(km=P16)):
        assert decode(L, c, s, **kw) == 1, kw
    assert decode(L, c, s, q=P16 + 2) == 8
    assert decode(L, c, s, ws=P16 + 16) == 8
    p = sage.SageDecodeParams(4, 0, 0, 0.0)
    n = L.sage_decode_workspace_bytes(ctypes.byref(c), ctypes.byref(s), ctypes.byref(p))
    assert n > 0 and decode(L, c, s, ws_bytes=n - 1) == 5
    tracked = cache(weight=P16)
    more = L.sage_decode_workspace_bytes(ctypes.byref(tracked), ctypes.byref(s), ctypes.byref(p))
    assert more >= n + 4 * 2 * 4 * 64  # a score for every query head and slot
    p.Hq = 3
    assert L.sage_decode_workspace_bytes(ctypes.byref(c), ctypes.byref(s), ctypes.byref(p)) == 0
    assert L.sage_attn_decode(P16, P16, None, None, None, None, None, P16, 1 << 30, None) == 1


def test_append_arguments(L):
    c, s = cache(), seqs()

    def append(k=P16, v=P16, n_new=None, km=None, T=1, layout=0):
        return L.sage_kv_append(k, v, n_new, km, T, layout, ctypes.byref(c), ctypes.byref(s), None)

    for kw in (dict(T=-1), dict(layout=2), dict(km=P16), dict(k=None), dict(v=None), dict(T=1 << 30)):
        assert append(**kw) == 1, kw
    assert append(k=P16 + 8) == 8 and append(n_new=P16 + 2) == 8


def test_evict_arguments(L):
    c, s = cache(weight=P16), seqs()

    def evict(dst=P16 + 64, pages=2, keep=32, sinks=4, recent=8, new_lens=P16 + 64, kept=P16, c=c):
        return L.sage_kv_evict(ctypes.byref(c), ctypes.byref(s), dst, pages, keep, sinks, recent, new_lens, kept, None)

    for kw in (dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=30), dict(pages=1), dict(pages=0),
               dict(dst=None), dict(new_lens=None), dict(kept=None), dict(dst=P16), dict(new_lens=P16),
               dict(c=cache())):
        assert evict(**kw) == 1, kw
    assert evict(kept=P16 + 2) == 8


def test_window_arguments(L):
    def fwd(q=P16, k=P16, v=P16, o=P16, lse=None, lens=None, **kw):
        base = dict(B=1, Hq=4, Hkv=2, N=100, d=64, dtype=0, layout=0, window=16, sinks=0, sm_scale=0.0)
        base.update(kw)
        p = sage.SageWindowParams(**base)
        return L.sage_attn_window_fwd(q, k, v, o, lse, lens, ctypes.byref(p), None)

    for kw in (dict(B=0), dict(Hq=3), dict(Hkv=0), dict(N=0), dict(layout=3), dict(window=-1), dict(sinks=-1),
               dict(sm_scale=float("nan")), dict(q=None), dict(o=None), dict(B=1 << 20, N=1 << 20)):
        assert fwd(**kw) == 1, kw
    assert fwd(d=80) == 2 and fwd(dtype=5) == 3
    assert fwd(q=P16 + 8) == 8 and fwd(lse=P16 + 2) == 8 and fwd(lens=P16 + 1) == 8
    assert L.sage_attn_window_fwd(P16, P16, P16, P16, None, None, None, None) == 1


# ---------------------------------------------------------------- the binding
def host_cache(**kw):
    return sage.KVCache.alloc(8, 16, 2, 64, device="cpu", **kw)


TABLE, LENS = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
BF = torch.bfloat16


def test_cache_construction():
    c = host_cache(quantized=True, track_weight=True, tensor_layout="NHD")
    assert c.k_pages.shape == (8, 16, 2, 64) and c.k_scale.shape == (8, 2, 16) and c.Hkv == 2 and c.page_size == 16
    k = torch.zeros((8, 2, 16, 64), dtype=BF)
    s = torch.zeros((8, 2, 16))
    for bad in (lambda: sage.KVCache(k, k[:4]), lambda: sage.KVCache(k, k.half()), lambda: sage.KVCache(k.float(), k.float()),
                lambda: sage.KVCache(k, k, s, s), lambda: sage.KVCache(k, k, tensor_layout="NDH"),
                lambda: sage.KVCache(k.transpose(1, 2), k.transpose(1, 2)), lambda: sage.KVCache(k[..., :32].contiguous(), k[..., :32].contiguous()),
                lambda: sage.KVCache(k[:, :, :8].contiguous(), k[:, :, :8].contiguous()),
                lambda: sage.KVCache(k.to(torch.int8), k.to(torch.float8_e4m3fn)),
                lambda: sage.KVCache(k, k, weight=s.half()), lambda: sage.KVCache(k[0], k[0])):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("kw", [dict(), dict(q=torch.zeros((2, 3, 64), dtype=BF)), dict(q=torch.zeros((1, 4, 64), dtype=BF)),
                                dict(q=torch.zeros((2, 4, 64), dtype=torch.float16)), dict(q=torch.zeros((2, 4, 64))),
                                dict(q=torch.zeros((2, 64, 4), dtype=BF).transpose(1, 2)), dict(window=-1),
                                dict(sinks=2 ** 31), dict(lens=LENS.long()), dict(lens=LENS[:1]),
                                dict(table=TABLE.T), dict(table=TABLE.long()), dict(out=torch.zeros((2, 4, 64))),
                                dict(workspace=torch.zeros(8))])
def test_decode_binding(kw):
    """Each call is refused; with good arguments (the first) because the tensors are on the CPU."""
    a = dict(q=torch.zeros((2, 4, 64), dtype=BF), table=TABLE, lens=LENS)
    a.update(kw)
    with pytest.raises(ValueError, match=None if kw else "CUDA device"):
        sage.sage_attn_decode(a.pop("q"), host_cache(), a.pop("table"), a.pop("lens"), **a)


def test_other_bindings():
    c, k = host_cache(track_weight=True), torch.zeros((2, 2, 3, 64), dtype=BF)
    dst = torch.ones((2, 2), dtype=torch.int32)
    km = torch.zeros((2, 2, 64))
    q = torch.zeros((1, 4, 50, 64), dtype=BF)
    calls = [lambda: sage.sage_kv_append(k, k, c, TABLE, LENS, km=km),
             lambda: sage.sage_kv_append(k, k[:, :, :2], c, TABLE, LENS),
             lambda: sage.sage_kv_append(k, k, c, TABLE, LENS, tensor_layout="NHD"),
             lambda: sage.sage_kv_append(k.half(), k.half(), c, TABLE, LENS),
             lambda: sage.sage_kv_append(k, k, c, TABLE, LENS, n_new=LENS.long()),
             lambda: sage.sage_kv_append(k, k, c, TABLE, LENS),
             lambda: sage.sage_attn_decode_lse(torch.zeros((2, 4, 64), dtype=BF), c, TABLE, LENS, km=km),
             lambda: sage.sage_kv_evict(host_cache(), TABLE, LENS, dst, 16),
             lambda: sage.sage_kv_evict(c, TABLE, LENS, dst, 33),
             lambda: sage.sage_kv_evict(c, TABLE, LENS, dst, 0),
             lambda: sage.sage_kv_evict(c, TABLE, LENS, dst, 16, sinks=10, recent=7),
             lambda: sage.sage_kv_evict(c, TABLE, LENS, dst, 16, kept=torch.zeros((2, 2, 8), dtype=torch.int32)),
             lambda: sage.sage_kv_evict(c, TABLE, LENS, dst, 16),
             lambda: sage.sage_attn_window_fwd(q, q, q, window=-1),
             lambda: sage.sage_attn_window_fwd(q, q[:, :, :40], q, window=8),
             lambda: sage.sage_attn_window_fwd(q, q, q.half(), window=8),
             lambda: sage.sage_attn_window_fwd(q.float(), q.float(), q.float(), window=8),
             lambda: sage.sage_attn_window_fwd(q.transpose(1, 2), q, q, window=8),
             lambda: sage.sage_attn_window_fwd(q, q, q, window=8, lens=LENS),
             lambda: sage.sage_attn_window_fwd(q, q, q, window=8, tensor_layout="NDH"),
             lambda: sage.sage_attn_window_fwd(q, q, q, window=8)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
