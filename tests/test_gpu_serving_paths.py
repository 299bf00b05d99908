"""Serving operators on the GPU where a call takes another way through them: the
ways of a decode (one CTA a row, or split and joined), prompts long enough for
the wide append, tiles of sinks, rows behind a sequence's end, alignments, calls
at the same time.  References and tolerances: tests/serving_ref.py."""
import math

import pytest
import torch

from quantized_attention_block_b200 import sage

from serving_ref import NAN, Paged, assert_within, decode_ref, evict_ref, quantize, window_ref
from test_gpu_serving import bits, check_decode, check_window, no_device_error, window_inputs  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ---------------------------------------------------------------- decode
@pytest.mark.parametrize("n", [511, 512, 513, 528])
@pytest.mark.parametrize("quantized", [False, True])
def test_decode_at_the_border_of_the_split(quantized, n):
    """32 blocks of 16 keys go to one CTA, 33 are split."""
    check_decode(Paged([n, 1, 200], 2, 64, BF, 16, quantized=quantized, weights=True), 8)


@pytest.mark.parametrize("longest", [2048, 2064])
def test_decode_many_rows_of_middling_length(longest):
    """Enough rows for every SM twice: up to 128 blocks a row to one CTA, more are split."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (150,), generator=g).tolist()
    lens[7], lens[149] = longest, 700
    check_decode(Paged(lens, 2, 64, FP, 16, weights=True), 4, hide=False)


def test_decode_without_a_join_needs_little_workspace():
    c = Paged([100, 30], 2, 64, BF, 16)
    cache, table, lens = c.to_gpu()
    n = sage.decode_workspace_bytes(cache, table, lens, 4)
    assert 0 < n <= 256
    ws = torch.full((n + 256,), 7, dtype=torch.uint8, device="cuda")[:n]
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(0)).to(BF)
    o = sage.sage_attn_decode(q.cuda(), cache, table, lens, workspace=ws)
    ref, _, to, _, _, _ = decode_ref(c, q)
    assert_within(o, ref, to)
    assert torch.equal(bits(o), bits(sage.sage_attn_decode(q.cuda(), cache, table, lens)))


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("n", [300, 1500])
def test_decode_8_bit_scales_of_every_size(order, n):
    """V whose rows' scales lie up to 2^200 apart, growing, falling and at random: the unit that the weights are
    held in moves with them, and nothing overflows or is lost next to the largest."""
    c = Paged([n], 2, 64, BF, 16, quantized=True)
    e = torch.linspace(-100, 100, n)
    e = e if order == "up" else e.flip(0) if order == "down" else e[torch.randperm(n, generator=torch.Generator().manual_seed(0))]
    g = torch.Generator().manual_seed(2)
    c.keys, c.values = [], []
    k = torch.randn((2, n, 64), generator=g).to(BF)
    v = (torch.randn((2, n, 64), generator=g) * torch.exp2(e)[:, None]).to(BF)
    v[1] = v[1] * 2.0 ** -100  # a head of small values only
    v[0, 5], v[1, 7] = 0, 0
    c.put(0, 0, k, v)
    q = torch.randn((1, 4, 64), generator=g).to(BF)
    cache, table, lens = c.to_gpu()
    o = sage.sage_attn_decode(q.cuda(), cache, table, lens)
    ref, _, _, _, _, err = decode_ref(c, q)
    for h in range(2):  # a tolerance for each head's own values
        top = c.values[0][h].abs().max().item()
        for x in (2 * h, 2 * h + 1):
            assert_within(o[0, x], ref[0, x], 2.0 ** -8 * ref[0, x].abs() + (4 * err + 2.0 ** -15) * top)


def test_decode_sequences_may_share_pages_and_calls_may_overlap():
    """Two sequences that read the same pages (a long row may be cut elsewhere, so the bytes may differ); calls on
    two streams at once, each with a workspace of its own, give what they give one after the other."""
    c = Paged([3000, 40], 4, 128, BF, 16)
    cache, table, lens = c.to_gpu()
    q = torch.randn((1, 8, 128), device="cuda").to(BF).expand(2, -1, -1).contiguous()
    both = torch.stack([table[0], table[0]]).contiguous()
    n = torch.full((2,), 3000, dtype=torch.int32, device="cuda")
    o = sage.sage_attn_decode(q, cache, both, n)
    ref, _, to, _, _, _ = decode_ref(c, q.cpu())
    assert_within(o[0], ref[0], to[0])
    assert_within(o[1], ref[0], to[0])
    want = [sage.sage_attn_decode(q, cache, table, lens, window=w) for w in (0, 2000)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for s, w, outs in zip(streams, (0, 2000), got):
            outs.append(sage.sage_attn_decode(q, cache, table, lens, window=w, stream=s))
    torch.cuda.synchronize()
    for outs, x in zip(got, want):
        assert all(torch.equal(bits(y), bits(x)) for y in outs)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("layout,in_layout", [("HND", "HND"), ("NHD", "HND"), ("HND", "NHD")])
@pytest.mark.parametrize("quantized", [False, True])
def test_append_long_ragged_prompts(quantized, layout, in_layout):
    """More rows than the wide form begins with; bit for bit, and nothing else changes."""
    B, H, T, d, page = 5, 8, 1301, 128, 32
    held, n_new = [0, 3, 100, 31, 64], [1301, 0, 640, 1300, 1]
    per = -(-(max(held) + T) // page)
    g = torch.Generator().manual_seed(0)
    cache = sage.KVCache.alloc(B * per + 2, page, H, d, BF, quantized=quantized, track_weight=True, tensor_layout=layout)
    cache.weight.fill_(3.0)
    table = torch.randperm(B * per + 2, generator=g)[:B * per].to(torch.int32).view(B, per)
    k, v = (3 * torch.randn((B, H, T, d), generator=g)).to(BF), torch.randn((B, H, T, d), generator=g).to(BF)
    kc, vc, ks, vs = quantize(k, v)
    if quantized:
        kc, vc = kc.view(torch.int8), vc.view(torch.int8)
    else:
        kc, vc = k, v
    want = [x.clone().cpu() for x in (cache.k_pages, cache.v_pages.view(torch.int8) if quantized else cache.v_pages)]
    extra = [x.clone().cpu() for x in ((cache.k_scale, cache.v_scale) if quantized else ())]
    weight = cache.weight.cpu()
    for b in range(B):
        pos = held[b] + torch.arange(n_new[b])
        at, row = table[b, pos // page].long(), pos % page
        for x, y in zip(want, (kc, vc)):
            (x.transpose(1, 2) if layout == "HND" else x)[at, row] = y[b, :, :n_new[b]].transpose(0, 1)
        for x, y in zip(extra, (ks, vs)):
            x.transpose(1, 2)[at, row] = y[b, :, :n_new[b]].transpose(0, 1)
        weight.transpose(1, 2)[at, row] = 0.0
    kk, vv = ((x if in_layout == "HND" else x.transpose(1, 2)).contiguous().cuda() for x in (k, v))
    sage.sage_kv_append(kk, vv, cache, table.cuda(), torch.tensor(held, dtype=torch.int32).cuda(),
                        n_new=torch.tensor(n_new, dtype=torch.int32).cuda(), tensor_layout=in_layout)
    got = [cache.k_pages, cache.v_pages.view(torch.int8) if quantized else cache.v_pages]
    got += [cache.k_scale, cache.v_scale] if quantized else []
    for x, y in zip(got, want + extra):
        assert torch.equal(bits(x.cpu()), bits(y))
    assert torch.equal(cache.weight.cpu(), weight)


# ---------------------------------------------------------------- evict
@pytest.mark.parametrize("fill", [0.0, -math.inf, math.inf, NAN])
def test_evict_equal_weights_keep_the_earliest(fill):
    c = Paged([3000], 2, 64, BF, 16, weights=True, spare=70)
    c.weight[:] = fill
    for j in (100, 1500, 2700):  # three that differ: lighter than infinity, heavier than the others
        pid, r = c.slot(0, j)
        c.weight[pid, 1, r] = 5.0
    cache, table, lens = c.to_gpu()
    _, kept = sage.sage_kv_evict(cache, table, lens, c.free[:63][None].contiguous().cuda(), 1000, sinks=5, recent=50)
    for h in range(2):
        w = [c.weight[c.slot(0, j)[0], h, c.slot(0, j)[1]] for j in range(3000)]
        assert kept[0, h].tolist() == evict_ref(w, 3000, 1000, 5, 50)


def test_evict_nothing_but_sinks_and_recent():
    c = Paged([500], 1, 64, BF, 16, weights=True, spare=10)
    cache, table, lens = c.to_gpu()
    new_lens, kept = sage.sage_kv_evict(cache, table, lens, c.free[:4][None].contiguous().cuda(), 60, sinks=20, recent=40)
    assert new_lens.tolist() == [60] and kept[0, 0].tolist() == list(range(20)) + list(range(460, 500))


# ---------------------------------------------------------------- window
@pytest.mark.parametrize("sinks", [1, 63, 64, 65, 127, 128, 129, 190, 256])
@pytest.mark.parametrize("window", [1, 65, 200])
def test_window_tiles_of_sinks(window, sinks):
    """Sinks that end in either half of a key tile, before, at and inside the window's own tiles."""
    q, k, v = window_inputs(1, 2, 1, 900, 64, BF, seed=sinks)
    check_window(q, k, v, window, sinks)


@pytest.mark.parametrize("window", [62, 63, 64, 65, 126, 129, 191, 193, 383])
@pytest.mark.parametrize("N", [448, 449, 577])
def test_window_starts_and_ends_in_either_half_of_a_tile(window, N):
    q, k, v = window_inputs(1, 1, 1, N, 128, FP, seed=window)
    check_window(q, k, v, window, 0)


def test_window_more_items_than_sms():
    """Several hundred heads: every item is taken once, from whichever CTA, with lengths that leave some out."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 301, (40,), generator=g).tolist()
    lens[3], lens[17], lens[39] = 0, 300, 257
    q, k, v = window_inputs(40, 12, 3, 300, 64, BF)
    check_window(q, k, v, 90, 3, lens=lens)


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_window_zeroes_rows_behind_the_end_in_tensors_it_makes(layout):
    """Rows behind a sequence's end: zeros in an output made by the call, untouched in one that is given."""
    lens = [0, 300, 513, 700, 1]
    q, k, v = window_inputs(5, 2, 2, 700, 64, BF)
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    qd, kd, vd = ((x if layout == "HND" else x.transpose(1, 2)).contiguous().cuda() for x in (q, k, v))
    junk = torch.full((64 << 20,), NAN, device="cuda")  # the allocator's next blocks hold NaN
    del junk
    o, lse = sage.sage_attn_window_fwd_lse(qd, kd, vd, window=100, sinks=2, lens=dl, tensor_layout=layout)
    mine = torch.full_like(o, -7.0)
    _, lse2 = sage.sage_attn_window_fwd_lse(qd, kd, vd, window=100, sinks=2, lens=dl, out=mine, tensor_layout=layout)
    given = torch.full_like(lse, -7.0)
    o2, _ = sage.sage_attn_window_fwd_lse(qd, kd, vd, window=100, sinks=2, lens=dl, lse=given, tensor_layout=layout)
    if layout == "NHD":
        o, o2, mine = (x.transpose(1, 2) for x in (o, o2, mine))
    for b, n in enumerate(lens):
        assert (o[b, :, n:] == 0).all() and (lse[b, :, n:] == 0).all() and (lse2[b, :, n:] == 0).all()
        assert (mine[b, :, n:] == -7).all() and (given[b, :, n:] == -7).all() and (o2[b, :, n:] == 0).all()
        assert torch.equal(bits(mine[b, :, :n]), bits(o[b, :, :n])) and torch.equal(given[b, :, :n], lse[b, :, :n])


@pytest.mark.parametrize("d", [64, 128])
def test_window_tensors_at_16_byte_boundaries(d):
    """Everything 16 bytes past a 256-byte boundary, and no byte next to the output changes."""
    q, k, v = window_inputs(2, 2, 1, 333, d, BF)

    def off(x):
        buf = torch.full((x.numel() + 16,), -7.0, dtype=x.dtype, device="cuda")
        y = buf[8:8 + x.numel()].view(x.shape)
        y.copy_(x)
        return buf, y

    (_, qd), (_, kd), (_, vd), (buf, out) = off(q), off(k), off(v), off(torch.zeros_like(q))
    assert out.data_ptr() % 32 == 16
    sage.sage_attn_window_fwd(qd, kd, vd, window=50, sinks=70, out=out)
    assert torch.equal(bits(out), bits(sage.sage_attn_window_fwd(q.cuda(), k.cuda(), v.cuda(), window=50, sinks=70)))
    assert (buf[:8] == -7).all() and (buf[-8:] == -7).all()


def test_window_rows_with_infinities_among_good_ones():
    """A value that is infinite for the rows that see it: those rows are computed apart, the others are not
    touched, and the bytes are the same every time."""
    q, k, v = window_inputs(1, 4, 2, 600, 128, BF)
    v[0, 0, 77, 3], v[0, 1, 300:340] = math.inf, NAN
    ref, _, to, _ = window_ref(q, torch.nan_to_num(k), torch.nan_to_num(v, nan=0.0, posinf=0.0), 60, 0)
    o = sage.sage_attn_window_fwd(q.cuda(), k.cuda(), v.cuda(), window=60)
    i = torch.arange(600)
    first, second = (i < 77) | (i >= 137), (i < 300) | (i >= 399)
    assert_within(o[:, :2, first], ref[:, :2, first], to[:, :2, first])
    assert_within(o[:, 2:, second], ref[:, 2:, second], to[:, 2:, second])
    assert torch.isinf(o[:, :2, ~first, 3]).all() and torch.isnan(o[:, 2:, ~second]).all()
    for _ in range(3):
        assert torch.equal(bits(o), bits(sage.sage_attn_window_fwd(q.cuda(), k.cuda(), v.cuda(), window=60)))


def test_window_calls_may_overlap():
    """Calls on two streams at once give what they give one after the other."""
    a = [x.cuda() for x in window_inputs(2, 8, 4, 1500, 128, BF)]
    b = [x.cuda() for x in window_inputs(3, 6, 6, 700, 64, FP)]
    want = [sage.sage_attn_window_fwd(*a, window=300, sinks=4), sage.sage_attn_window_fwd(*b, window=0)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        got[0].append(sage.sage_attn_window_fwd(*a, window=300, sinks=4, stream=streams[0]))
        got[1].append(sage.sage_attn_window_fwd(*b, window=0, stream=streams[1]))
    torch.cuda.synchronize()
    for outs, x in zip(got, want):
        assert all(torch.equal(bits(y), bits(x)) for y in outs)
