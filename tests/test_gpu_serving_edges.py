"""Serving operators on the GPU at the edges of their number formats and of what
their inputs may hold.  References in 64 bits; tolerances are counted in the test."""
import math

import pytest
import torch

from quantized_attention_block_b200 import sage

from serving_ref import HALF_STEP, assert_within, out_tol, score_error
from test_gpu_serving import no_device_error  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
LN2 = math.log(2.0)


# ---------------------------------------------------------------- light keys beside a heavy one
@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("d,dtype", [(64, FP), (128, FP), (64, BF)])
@pytest.mark.parametrize("B,H,n", [(37, 8, 2048), (1, 1, 8192)])
def test_decode_keeps_light_keys_beside_heavy_ones(B, H, n, d, dtype, G):
    """A heavy key with V = 0 in the first block of each warp, the others 2^-25 as heavy: all of the output comes from
    them.  Rows that one CTA does alone (128 blocks), and a split one (shares of 8 blocks)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    per = n // 16
    t = -25.0 + torch.randint(-32, 33, (B, H, n), generator=g, device="cuda") / 64.0
    v = 512.0 + 1024.0 * torch.rand((B, H, n, d), generator=g, device="cuda")
    at = torch.arange(per, device="cuda")
    heavy = (at[at % 8 < 4] if B == 1 else at[:4]) * 16
    t[..., heavy], v[..., heavy, :] = 0.0, 0.0
    if dtype == BF:
        t = t.round()  # (bf16 holds eight bits of a score)
    k = torch.zeros((B, H, n, d), device="cuda")
    k[..., 0] = t
    k, v = k.to(dtype), v.to(dtype)
    q = torch.randn((B, H * G, d), generator=g, device="cuda").to(dtype)
    q[..., 0] = 1.0

    def pages(x):
        return x.view(B, H, per, 16, d).transpose(1, 2).reshape(B * per, H, 16, d).contiguous()

    cache = sage.KVCache(pages(k), pages(v))
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    got, lse = sage.sage_attn_decode_lse(q, cache, table, lens, sm_scale=LN2)
    p = torch.exp2(t.double())
    l = p.sum(-1, keepdim=True)
    ref = ((p / l)[..., None] * v.double()).sum(2)[:, :, None].expand(-1, -1, G, -1).reshape(B, H * G, d)
    # Scores off by err move a weight by a factor e^(+-2 err), here of an output without the heavy key's V; the two
    # 16-bit parts of a weight carry 16 bits, or (fp16, which ends at 2^-24) half of 2^-24 x 2^-15 of the warp's
    # heaviest; exponentials 2^-22; a warp and turn rounds its sum once (or truncates: 2^-23), then pieces are joined.
    err = score_error(torch.ones(1, 1), torch.full((1, 1), 26.0), LN2) + 2.0 ** -22
    rel = 4 * err + 2.0 ** -16 + 2.0 ** -22 + (n / 64 + 600) * 2.0 ** -23
    tol = (HALF_STEP[dtype] + rel) * ref + n * 2.0 ** -40 / l[..., 0].min().item() * v.abs().max().item() + 2.0 ** -25
    assert (ref > 2.0 ** -14).all()
    assert ((got.double() - ref).abs() <= tol).all(), ((got.double() / ref).min().item(), (got.double() / ref).max().item())
    want = torch.log(l[..., 0])[:, :, None].expand(-1, -1, G).reshape(B, H * G)
    assert ((lse.double() - want).abs() <= err + 2.0 ** -21 * (4 + want.abs())).all()


@pytest.mark.parametrize("window", [0, 900])
@pytest.mark.parametrize("d,dtype", [(64, FP), (128, FP), (128, BF)])
def test_window_keeps_light_keys_beside_a_heavy_one(window, d, dtype):
    """Key 0 (a sink) with V = 0, the others 2^-24.5 as heavy: fp16 ends at 2^-24 of what a weight is a part of."""
    N, light = 1500, -24.5
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros((1, 1, N, d), device="cuda")
    k[..., 0] = light
    k[..., 0, 0] = 0.0
    v = 512.0 + 1024.0 * torch.rand((1, 1, N, d), generator=g, device="cuda")
    v[..., 0, :] = 0.0
    q = torch.randn((1, 1, N, d), generator=g, device="cuda")
    q[..., 0] = 1.0
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    got, lse = sage.sage_attn_window_fwd_lse(q, k, v, window=window, sinks=1, sm_scale=LN2)
    i = torch.arange(N, device="cuda")
    see = (i[None] <= i[:, None]) & ((i[:, None] - i[None] < window) | (i[None] < 1) | (window == 0))
    p = torch.exp2(k[0, 0, :, 0].double()) * see
    l = p.sum(-1, keepdim=True)
    ref = (p / l) @ v[0, 0].double()
    # The weights in the inputs' type: half a step, and as much again for their sum (taken before that rounding); in
    # fp16 at least half of 2^-24, in units of at most 2^-7 of the heaviest.  The rest as above; steps of 64 keys are
    # four products of 16.
    err = score_error(torch.ones(1, 1), torch.full((1, 1), 25.0), LN2) + 2.0 ** -22
    rel = 3 * HALF_STEP[dtype] + 4 * err + 2.0 ** -21 + (N / 16 + 8) * 2.0 ** -23
    tol = rel * ref + 2.0 ** -25 + (N * 2.0 ** -32 * v.abs().max().item() if dtype == FP else 0.0)
    got = got[0, 0].double()
    assert ((got - ref).abs() <= tol).all(), (got[-1] / ref[-1]).mean().item()
    assert ((lse[0, 0].double() - torch.log(l[:, 0])).abs() <= err + 2.0 ** -21 * (4 + torch.log(l[:, 0]).abs())).all()


# ---------------------------------------------------------------- NaN and infinity in V, in many items
@pytest.fixture
def short_waits():
    """Waits inside the kernels give up after 20 ms; what they wait for here takes microseconds."""
    sage.sage_debug_wait_limit(20000)
    yield
    torch.cuda.synchronize()
    sage.sage_debug_wait_limit(0)


def some_rows(q, k, v, b, h, rows, window, sinks):
    """(o, tolerance) of some rows of a head in 64 bits, over their visible keys alone."""
    hk = h // (q.shape[1] // k.shape[1])
    qq, kk = q[b, h, rows].double().cpu(), k[b, hk].double().cpu()
    scale = 1.0 / math.sqrt(q.shape[-1])
    o, tol = [], []
    for x, i in zip(qq, rows.tolist()):
        j = torch.arange(i + 1)
        j = j if window == 0 else j[(i - j < window) | (j < sinks)]
        vv = v[b, hk, j].double().cpu()
        w = torch.softmax(kk[j] @ x * scale, 0)
        o.append(w @ vv)
        # as in serving_ref.window_ref
        finite = torch.nan_to_num(vv, nan=0.0, posinf=0.0, neginf=0.0).abs()
        tol.append(out_tol(o[-1], finite, score_error(x[None], kk[j], scale), q.dtype)
                   + 2 * HALF_STEP[q.dtype] * (w @ finite))
    return torch.stack(o), torch.stack(tol)


def many_items(N, d, dtype, H, Hkv):
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((1, h, N, d), generator=g, device="cuda").to(dtype) for h in (H, Hkv, Hkv))
    return q, k, v


@pytest.mark.parametrize("d,dtype,window", [(128, BF, 0), (64, FP, 0), (128, FP, 300)])
def test_window_a_visible_infinity_reaches_its_channel_alone(short_waits, d, dtype, window):
    """An infinity in the V of key 0, which every row sees: seven items a CTA, none of which is held up."""
    q, k, v = many_items(8192, d, dtype, 32, 8)
    want, want_lse = sage.sage_attn_window_fwd_lse(q, k, v, window=window, sinks=1)
    v[:, :, 0, 3] = math.inf
    got, lse = sage.sage_attn_window_fwd_lse(q, k, v, window=window, sinks=1)
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 0
    assert (got[..., 3] == math.inf).all()
    keep = [c for c in range(d) if c != 3]
    assert torch.equal(got[..., keep], want[..., keep]) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("d,dtype", [(128, BF), (64, FP)])
def test_window_a_late_nan_leaves_the_rows_before_it(short_waits, d, dtype):
    q, k, v = many_items(8192, d, dtype, 32, 8)
    want = sage.sage_attn_window_fwd(q, k, v, window=0)
    v[:, :, 5000, 3] = math.nan
    got = sage.sage_attn_window_fwd(q, k, v, window=0)
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 0
    assert torch.equal(got[:, :, :4992], want[:, :, :4992])  # row tiles that do not reach key 5000
    keep = [c for c in range(d) if c != 3]
    assert torch.equal(got[:, :, 5000:][..., keep], want[:, :, 5000:][..., keep])
    assert torch.isnan(got[:, :, 5000:, 3]).all()
    for h in (0, 13, 31):
        ref, tol = some_rows(q, k, v, 0, h, torch.arange(4992, 5000), 0, 0)
        assert_within(got[0, h, 4992:5000], ref, tol)


@pytest.mark.parametrize("d,dtype,window,sinks", [(128, BF, 0, 0), (64, FP, 700, 70)])
def test_window_nan_in_every_value_of_a_channel(short_waits, d, dtype, window, sinks):
    """Nearly every row is computed again: thousands of them, none within a wait of another role."""
    q, k, v = many_items(4096, d, dtype, 32, 32)
    v[..., 3] = math.nan
    got = sage.sage_attn_window_fwd(q, k, v, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 0
    assert torch.isnan(got[..., 3]).all()
    keep = [c for c in range(d) if c != 3]
    assert torch.isfinite(got[..., keep]).all()
    rows = torch.tensor([0, 1, 63, 127, 128, 700, 1999, 2048, 3333, 4095])
    for h in (0, 17, 31):
        ref, tol = some_rows(q, k, v, 0, h, rows, window, sinks)
        assert_within(got[0, h, rows][..., keep], ref[:, keep], tol[:, keep])


# ---------------------------------------------------------------- errors
def test_a_timeout_does_not_hide_a_bad_page():
    cache = sage.KVCache.alloc(8, 16, 2, 64, BF)
    table = torch.full((1, 2), 99, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 20, dtype=torch.int32, device="cuda")
    sage.sage_attn_decode(torch.zeros((1, 4, 64), dtype=BF, device="cuda"), cache, table, lens)
    assert sage.sage_debug_bounded_wait(2000) == 7
    assert [sage.sage_last_device_error() for _ in range(2)] == [9, 0]


# ---------------------------------------------------------------- padded batches
@pytest.mark.parametrize("max_pages", [2, 100])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_decode_of_an_empty_sequence_goes_by_its_length_alone(bad, max_pages):
    """Without a key, o = 0 and lse = -inf, whatever the row's query and km hold; one CTA a row, and split."""
    cache = sage.KVCache.alloc(8, 16, 2, 64, BF, quantized=True)
    table = torch.zeros((3, max_pages), dtype=torch.int32, device="cuda")
    table[1, :2] = torch.tensor([3, 4])
    lens = torch.tensor([0, 20, 0], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((3, 2, 20, 64), generator=g, device="cuda").to(BF) for _ in range(2))
    sage.sage_kv_append(k, v, cache, table, torch.zeros_like(lens), n_new=lens)
    q = torch.randn((3, 4, 64), generator=g, device="cuda").to(BF)
    km = torch.randn((3, 2, 64), generator=g, device="cuda")
    want = sage.sage_attn_decode_lse(q, cache, table, lens, km=km)
    q[0], q[2], km[2] = bad, bad, bad
    o, lse = sage.sage_attn_decode_lse(q, cache, table, lens, km=km)
    assert (o[[0, 2]] == 0).all() and (lse[[0, 2]] == -math.inf).all()
    assert torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1]) and torch.isfinite(lse[1]).all()


# ---------------------------------------------------------------- largest arguments
def test_evict_to_the_largest_budget():
    """keep = 2^31 - 1: every token stays, the 8 GB of kept end in -1, and nothing before them is written."""
    keep, page = 2 ** 31 - 1, 1024
    cache = sage.KVCache.alloc(2, page, 1, 64, BF, track_weight=True)
    cache.k_pages[0] = torch.randn((1, page, 64), device="cuda").to(BF)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    dst = torch.full((1, -(-keep // page)), -1, dtype=torch.int32, device="cuda")
    dst[0, 0] = 1
    lens = torch.full((1,), 700, dtype=torch.int32, device="cuda")
    buf = torch.full((keep + 4097,), 7, dtype=torch.int32, device="cuda")
    at = 4096 - 3  # (not aligned to more than its type)
    kept = buf[at:at + keep].view(1, 1, keep)
    new_lens, _ = sage.sage_kv_evict(cache, table, lens, dst, keep, sinks=4, recent=16, kept=kept)
    assert new_lens.tolist() == [700]
    assert torch.equal(kept[0, 0, :700], torch.arange(700, dtype=torch.int32, device="cuda"))
    assert kept[0, 0, 700:].amin() == -1 == kept[0, 0, 700:].amax()
    assert (buf[:at] == 7).all() and (buf[at + keep:] == 7).all()
    assert torch.equal(cache.k_pages[1, 0, :700], cache.k_pages[0, 0, :700])
    assert not cache.k_pages[1, 0, 700:].any()
