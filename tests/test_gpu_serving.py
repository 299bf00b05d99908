"""The serving operators on the GPU against their plain 64-bit forms
(tests/serving_ref.py): the paged cache, attention of one new token, eviction,
sliding-window attention, and a run of them together.  Every slot that a call
must not look at holds NaN."""
import math

import pytest
import torch

from quantized_attention_block_b200 import sage

from serving_ref import (NAN, Paged, assert_within, decode_ref, evict_ref, quantize, visible, window_ref)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 0


def bits(t):
    return t.contiguous().view(torch.uint8)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("in_layout", ["HND", "NHD"])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("d,dtype,quantized,use_km", [(64, BF, False, False), (128, FP, False, False),
                                                      (64, FP, True, True), (128, BF, True, False),
                                                      (128, BF, True, True)])
def test_append(d, dtype, quantized, use_km, layout, in_layout):
    """Codes, scales and copies bit for bit; every other byte of the pool as it was."""
    held, n_new, T, H, page = [0, 5, 31, 100, 16], [7, 0, 33, 40, 1], 40, 3, 16
    c = Paged(held, H, d, dtype, page, quantized=quantized, layout=layout, extra=T, weights=True)
    cache, table, lens = c.to_gpu()
    g = torch.Generator().manual_seed(1)
    k, v = ((4 * torch.randn((5, H, T, d), generator=g)).to(dtype) for _ in range(2))
    k[0, 0, 1] = 0  # a zero row has scale 0 and codes 0
    v[0, 1, 2] = 0
    k[2, 1, 3, 5], v[3, 2, 4, 6] = NAN, NAN
    km = torch.randn((5, H, d), generator=g) if use_km else None
    if use_km:
        k[0, 0, 1] = 0
    kk, vv = ((x if in_layout == "HND" else x.transpose(1, 2).contiguous()).cuda() for x in (k, v))
    want = [x.clone().cpu() for x in (cache.k_pages, cache.v_pages.view(torch.int8) if quantized else cache.v_pages)]
    ws = [cache.k_scale.cpu(), cache.v_scale.cpu()] if quantized else []
    weight = cache.weight.cpu()
    for b in range(5):
        kc, vc, ks, vs = quantize(k[b], v[b], None if km is None else km[b][:, None])
        if not quantized:
            kc, vc = k[b], v[b]
        for i in range(n_new[b]):
            pid, r = c.slot(b, held[b] + i)
            at = (pid, slice(None), r) if layout == "HND" else (pid, r)
            want[0][at] = kc[:, i]
            want[1][at] = vc.view(torch.int8)[:, i] if quantized else vc[:, i]
            if quantized:
                ws[0][pid, :, r], ws[1][pid, :, r] = ks[:, i], vs[:, i]
            weight[pid, :, r] = 0.0
    sage.sage_kv_append(kk, vv, cache, table, lens, n_new=torch.tensor(n_new, dtype=torch.int32).cuda(),
                        km=None if km is None else km.cuda(), tensor_layout=in_layout)
    torch.cuda.synchronize()
    got = [cache.k_pages.cpu(), (cache.v_pages.view(torch.int8) if quantized else cache.v_pages).cpu()]
    if quantized:
        for x, y in zip((cache.k_scale.cpu(), cache.v_scale.cpu()), ws):
            assert torch.equal(torch.isnan(x), torch.isnan(y))
            assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))
        bad = torch.isnan(ws[0]), torch.isnan(ws[1])  # a NaN row's codes are any; its scale says NaN
        for x, y, nan in zip(got, want, bad):
            nan = nan[..., None] if layout == "HND" else nan.transpose(1, 2)[..., None]
            assert torch.equal(x.masked_fill(nan, 0), y.masked_fill(nan, 0))
    else:
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, want))
    assert torch.equal(cache.weight.cpu(), weight)


def test_append_nothing_and_past_the_end():
    c = Paged([30, 16], 2, 64, BF, 16, extra=2)
    cache, table, lens = c.to_gpu()
    k = torch.ones((2, 2, 0, 64), dtype=BF, device="cuda")
    before = bits(cache.k_pages).clone()
    sage.sage_kv_append(k, k, cache, table, lens)
    assert torch.equal(bits(cache.k_pages), before)
    assert sage.sage_last_device_error() == 0
    # sequence 0 has room for two tokens, sequence 1's second page is no page: one error, no write elsewhere
    table[1, 1] = c.n_pages
    k = torch.ones((2, 2, 3, 64), dtype=BF, device="cuda")
    sage.sage_kv_append(k, k, cache, table, lens)
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 9 and sage.sage_last_device_error() == 0
    page = cache.k_pages[int(c.table[0, 1])].cpu()
    assert torch.equal(page[:, 14:], torch.ones_like(page[:, 14:]))
    changed = (bits(cache.k_pages) != before).view(c.n_pages, -1).any(1).nonzero().flatten().tolist()
    assert changed == [int(c.table[0, 1])]


# ---------------------------------------------------------------- decode
def check_decode(c: Paged, Hq, window=0, sinks=0, scale=None, seed=3, hide=True, km=False):
    g = torch.Generator().manual_seed(seed)
    B = len(c.lens)
    q = torch.randn((B, Hq, c.d), generator=g).to(c.dtype)
    o, lse, to, tl, grown, err = decode_ref(c, q, window, sinks, scale)
    if hide:
        for b, n in enumerate(c.lens):
            seen = set(visible(n - 1, n, window, sinks).tolist()) if n else set()
            c.hide(b, [j for j in range(n) if j not in seen])
    cache, table, lens = c.to_gpu()
    kmt = torch.randn((B, c.Hkv, c.d), generator=g) if km else None
    if km:
        s = scale or 1 / math.sqrt(c.d)
        dot = torch.einsum("bhgd,bhd->bhg", q.double().view(B, c.Hkv, -1, c.d), kmt.double()).reshape(B, Hq) * s
        lse = lse + dot
        tl = tl + 2.0 ** -19 * (1 + dot.abs()) + 2.0 ** -22 * (q.double().abs() @ torch.ones(c.d).double()) * 4 * s
    # the outputs between sentinels: no byte outside of them changes
    buf = torch.full((q.numel() + 2048,), -7.0, dtype=c.dtype, device="cuda")
    out = buf[1024:1024 + q.numel()].view(q.shape)
    got, got_lse = sage.sage_attn_decode_lse(q.cuda(), cache, table, lens, window=window, sinks=sinks, sm_scale=scale,
                                             km=None if kmt is None else kmt.cuda(), out=out)
    torch.cuda.synchronize()
    assert torch.equal(buf[:1024], torch.full_like(buf[:1024], -7.0)) and torch.equal(buf[-1024:], torch.full_like(buf[:1024], -7.0))
    assert_within(got, o, to, "o")
    assert_within(got_lse, lse, tl, "lse")
    if c.weight is not None:
        want, tol = c.weight.double().clone(), torch.zeros(c.weight.shape, dtype=torch.float64)
        G = Hq // c.Hkv
        for b, at_p in enumerate(grown):
            if at_p is None:
                continue
            for j, p in zip(at_p[0].tolist(), at_p[1].T):
                pid, r = c.slot(b, j)
                want[pid, :, r] += p
                # each head's weight off by a factor e^(+-2 err) and a few fp32 roundings
                tol[pid, :, r] = (2.1 * err + 2.0 ** -19) * p + G * 2.0 ** -23 * want[pid, :, r].abs()
        assert_within(cache.weight, want, tol, "weight")
    # the same bytes again (the weights do not enter)
    again = sage.sage_attn_decode(q.cuda(), cache, table, lens, window=window, sinks=sinks, sm_scale=scale)
    assert torch.equal(bits(again), bits(got))
    return got


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 1000, 0, 333]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (16, 16), (17, 1), (100, 40), (100, 200), (5000, 9)])
@pytest.mark.parametrize("d,dtype,quantized", [(64, BF, False), (128, FP, False), (64, FP, True), (128, BF, True)])
def test_decode_masks(d, dtype, quantized, window, sinks):
    check_decode(Paged(LENS, 2, d, dtype, 16, quantized=quantized, weights=True), 6, window, sinks)


@pytest.mark.parametrize("G", [1, 2, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("d,dtype,quantized,layout,page", [(128, BF, False, "HND", 64), (64, FP, False, "NHD", 16),
                                                           (128, FP, True, "NHD", 32), (64, BF, True, "HND", 1024)])
def test_decode_head_groups(d, dtype, quantized, layout, page, G):
    check_decode(Paged([77, 300], 3, d, dtype, page, quantized=quantized, layout=layout, weights=G in (5, 17)), 3 * G,
                 km=quantized, window=200 if G == 2 else 0, sinks=3 if G == 2 else 0)


@pytest.mark.parametrize("H,B,hi", [(1, 1, 9000), (1, 3, 5000), (2, 300, 90), (5, 130, 40)])
def test_decode_splits(H, B, hi):
    """One long row over every CTA; more sequences than a CTA's threads, empty ones among them."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, hi, (B,), generator=g).tolist()
    lens[0], lens[-1] = hi, hi
    if B > 100:
        lens[1:9] = [0] * 8
        lens[-9:-1] = [0] * 8
    check_decode(Paged(lens, H, 64, BF, 16, weights=B == 3), 4 * H, hide=False)


def test_decode_scale_and_all_empty():
    check_decode(Paged([40, 70], 2, 128, BF, 16), 4, scale=0.3)
    check_decode(Paged([0, 0, 0], 2, 128, BF, 16), 4)


@pytest.mark.parametrize("quantized", [False, True])
def test_decode_visible_nan_stays_in_its_sequence(quantized):
    c = Paged([50, 50, 50], 2, 64, BF, 16, quantized=quantized)
    pid, r = c.slot(1, 20)
    c.k[pid, 0, r, 3], c.ks[pid, 0, r] = NAN, NAN
    cache, table, lens = c.to_gpu()
    q = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(0)).to(BF)
    o, lse = sage.sage_attn_decode_lse(q.cuda(), cache, table, lens)
    assert torch.isnan(o[1, :2]).all() and torch.isnan(lse[1, :2]).all()
    ref, rl, to, tl, _, _ = decode_ref(c, q)
    for at in ((0, slice(None)), (2, slice(None)), (1, slice(2, 4))):
        assert_within(o[at], ref[at], to[at])


def test_decode_bad_pages_and_lengths():
    """A page number outside the pool counts as a page without tokens, a length outside the table as the
    nearest bound; both are reported once.  Nothing is read out of bounds: the kernel checks each number."""
    c = Paged([100, 100, 40], 2, 64, BF, 16, seed=5, weights=True)
    q = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(0)).to(BF)
    cache, table, lens = c.to_gpu()
    table[0, 2], table[0, 6] = -1, c.n_pages
    lens[2] = -5
    o, lse = sage.sage_attn_decode_lse(q.cuda(), cache, table, lens)
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 9 and sage.sage_last_device_error() == 0
    gone = torch.tensor([j not in range(32, 48) and j < 96 for j in range(100)])
    c.keys[0], c.values[0] = c.keys[0][:, gone], c.values[0][:, gone]
    c.lens = [int(gone.sum()), 100, 0]
    ref, rl, to, tl, _, _ = decode_ref(c, q)
    assert_within(o, ref, to)
    assert_within(lse, rl, tl)
    # entries behind the visible keys are not looked up
    c = Paged([100], 2, 64, BF, 16)
    cache, table, lens = c.to_gpu()
    table[0, 1:4] = -1  # a window of 30 sees tokens 70 on, and the sink in page 0
    sage.sage_attn_decode(q[:1].cuda(), cache, table, lens, window=30, sinks=4)


def test_decode_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements in K and in V."""
    H, d, page = 8, 128, 64
    n_pages = 2 ** 31 // (H * d * page) + 100
    c = Paged([500, 77], H, d, BF, page)
    cache, table, lens = c.to_gpu()
    big = torch.empty((n_pages, H, page, d), dtype=BF, device="cuda")
    big_v = torch.empty_like(big)
    to = torch.arange(n_pages - c.n_pages, n_pages, device="cuda")
    big[to], big_v[to] = cache.k_pages, cache.v_pages
    far = torch.where((table >= 0) & (table < c.n_pages), table + (n_pages - c.n_pages), table).to(torch.int32)
    q = torch.randn((2, 8, d), generator=torch.Generator().manual_seed(0)).to(BF)
    got = sage.sage_attn_decode(q.cuda(), sage.KVCache(big, big_v), far, lens)
    assert torch.equal(bits(got), bits(sage.sage_attn_decode(q.cuda(), cache, table, lens)))
    k = torch.full((2, H, 1, d), 5.0, dtype=BF, device="cuda")
    sage.sage_kv_append(k, k, sage.KVCache(big, big_v), far, lens - 1)
    torch.cuda.synchronize()
    assert (big[int(far[0, 499 // page]), :, 499 % page] == 5.0).all()


def test_decode_graphs_share_a_workspace_and_streams():
    """Two captured graphs with one workspace, replayed with other lengths, and a call on another stream."""
    c = Paged([900, 33, 500], 2, 128, BF, 16, weights=True)
    cache, table, lens = c.to_gpu()
    q = torch.randn((3, 8, 128), device="cuda").to(BF)
    n = max(sage.decode_workspace_bytes(cache, table, lens, 8), sage.decode_workspace_bytes(cache, table, lens, 8, window=64))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    windows = (0, 64)
    for g, o, w in zip(graphs, outs, windows):
        sage.sage_attn_decode(q, cache, table, lens, window=w, out=o, workspace=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            sage.sage_attn_decode(q, cache, table, lens, window=w, out=o, workspace=ws)
    for new in ([900, 33, 500], [1, 0, 77], [899, 32, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for o, w in zip(outs, windows):
            want = sage.sage_attn_decode(q, cache, table, lens, window=w)
            other = sage.sage_attn_decode(q, cache, table, lens, window=w, stream=side)
            side.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(bits(o), bits(want)) and torch.equal(bits(other), bits(want))


# ---------------------------------------------------------------- evict
@pytest.mark.parametrize("quantized,layout,d,dtype,page", [(False, "HND", 128, BF, 16), (False, "NHD", 64, FP, 32),
                                                           (True, "HND", 128, FP, 64), (True, "NHD", 64, BF, 16)])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (40, 4, 10), (40, 0, 40), (100, 16, 0), (2000, 4, 4)])
def test_evict(quantized, layout, d, dtype, page, keep, sinks, recent):
    lens = [0, 1, 40, 41, 700, 1500, 99]
    H = 2
    per = -(-keep // page)
    c = Paged(lens, H, d, dtype, page, quantized=quantized, layout=layout, weights=True, spare=len(lens) * per + 2)
    for b, n in enumerate(lens):  # ties, infinities, NaN, both zeros, negative numbers
        for j in range(n):
            pid, r = c.slot(b, j)
            if b == 3:
                c.weight[pid, :, r] = 1.0
            elif b in (4, 6):
                c.weight[pid, 0, r] = float(j % 7) - 2.0
                if j % 5 == 0:
                    c.weight[pid, 1, r] = NAN
                elif j % 11 == 0:
                    c.weight[pid, 1, r] = math.inf
                elif j % 13 == 0:
                    c.weight[pid, 1, r] = -0.0 if j % 2 else 0.0
    cache, table, dlens = c.to_gpu()
    dst = c.free[:len(lens) * per].view(len(lens), per)
    before = [x.clone() for x in (cache.k_pages, cache.v_pages.view(torch.uint8) if quantized else cache.v_pages)]
    scales = [x.clone() for x in (cache.weight, cache.k_scale, cache.v_scale) if x is not None]
    new_lens, kept = sage.sage_kv_evict(cache, table, dlens, dst.cuda(), keep, sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    want, want_s = [x.cpu() for x in before], [x.cpu() for x in scales]
    for b, n in enumerate(lens):
        for h in range(H):
            w = [c.weight[c.slot(b, j)[0], h, c.slot(b, j)[1]] for j in range(n)]
            stay = evict_ref(w, n, keep, sinks, recent)
            assert kept[b, h].tolist() == stay + [-1] * (keep - len(stay)), (b, h)
            for i, j in enumerate(stay):
                (sp, sr), (dp, dr) = c.slot(b, j), (int(dst[b, i // page]), i % page)
                for x in want:
                    if layout == "HND":
                        x[dp, h, dr] = x[sp, h, sr]
                    else:
                        x[dp, dr, h] = x[sp, sr, h]
                for x in want_s:
                    x[dp, h, dr] = x[sp, h, sr]
    got = [cache.k_pages, cache.v_pages.view(torch.uint8) if quantized else cache.v_pages]
    got_s = [x for x in (cache.weight, cache.k_scale, cache.v_scale) if x is not None]
    for x, y in zip(got + got_s, want + want_s):
        assert torch.equal(bits(x.cpu()), bits(y))


def test_evict_many_rows_and_long():
    """More rows than SMs, and a long row with few distinct weights."""
    for B, H, n, page, keep in ((40, 8, 50, 16, 20), (1, 1, 70000, 64, 30000)):
        per = -(-keep // page)
        pool = -(-n // page) * B
        g = torch.Generator(device="cuda").manual_seed(0)
        k = torch.randn((pool + per * B, H, page, 64), generator=g, device="cuda").to(BF)
        cache = sage.KVCache(k, k.clone(), weight=torch.randint(0, 50, k.shape[:3], generator=g, device="cuda").float())
        pages = torch.randperm(pool + per * B, generator=g, device="cuda").to(torch.int32)
        table, dst = pages[:pool].view(B, -1).contiguous(), pages[pool:].view(B, -1).contiguous()
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        w = cache.weight[table.long()].transpose(1, 2).reshape(B, H, -1)[..., :n].cpu()
        _, kept = sage.sage_kv_evict(cache, table, lens, dst, keep, sinks=2, recent=5)
        kept = kept.cpu()
        for b in range(0, B, 7):
            for h in range(0, H, 3):
                order = torch.sort(-w[b, h, 2:n - 5], stable=True)[1][:keep - 7] + 2
                want = torch.cat([torch.arange(2), torch.sort(order)[0], torch.arange(n - 5, n)])
                assert torch.equal(kept[b, h].long(), want)
        i = torch.tensor([0, 1, keep // 2, keep - 1])
        src = kept[0, 0, i].long()
        assert torch.equal(cache.k_pages[dst[0, i // page].long(), 0, i % page],
                           cache.k_pages[table[0, src // page].long(), 0, src % page])


def test_evict_bad_page():
    c = Paged([100], 2, 64, BF, 16, weights=True, spare=8)
    cache, table, lens = c.to_gpu()
    dst = c.free[:2][None].clone().cuda()
    dst[0, 1] = c.n_pages + 3
    table[0, 3] = -2
    before = bits(cache.k_pages).clone()
    sage.sage_kv_evict(cache, table, lens, dst, 32)
    torch.cuda.synchronize()
    assert sage.sage_last_device_error() == 9 and sage.sage_last_device_error() == 0
    changed = (bits(cache.k_pages) != before).view(c.n_pages, -1).any(1).nonzero().flatten().tolist()
    assert changed == [int(c.free[0])]


# ---------------------------------------------------------------- window
def window_inputs(B, Hq, Hkv, N, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((B, H, N, d), generator=g) for H in (Hq, Hkv, Hkv))
    k += 2.0 * torch.randn((1, Hkv, 1, d), generator=g)
    return q.to(dtype), k.to(dtype), v.to(dtype)


def check_window(q, k, v, window, sinks, lens=None, layout="HND", scale=None):
    B, Hq, N, d = q.shape
    ref, rl, to, tl = window_ref(q, k, v, window, sinks, lens, scale)
    q, k, v = (x.clone() for x in (q, k, v))
    if lens is not None:
        for b, n in enumerate(lens):
            for x in (q, k, v):
                x[b, :, n:] = NAN
    qd, kd, vd = ((x if layout == "HND" else x.transpose(1, 2)).contiguous().cuda() for x in (q, k, v))
    buf = torch.full((q.numel() + 2048,), -7.0, dtype=q.dtype, device="cuda")
    out = buf[1024:1024 + q.numel()].view(qd.shape)
    lse = torch.full((B, Hq, N), -7.0, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    sage.sage_attn_window_fwd_lse(qd, kd, vd, window=window, sinks=sinks, lens=dl, out=out, lse=lse, sm_scale=scale,
                                  tensor_layout=layout)
    torch.cuda.synchronize()
    out = out if layout == "HND" else out.transpose(1, 2)
    live = ~torch.isnan(rl)
    assert (out.cpu()[~live] == -7.0).all() and (lse.cpu()[~live] == -7.0).all()  # rows behind the end: as they were
    assert (buf[:1024] == -7.0).all() and (buf[-1024:] == -7.0).all()
    assert_within(out.cpu()[live], ref[live], to[live], "o")
    assert_within(lse.cpu()[live], rl[live], tl[live], "lse")


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 255, 257, 500])
@pytest.mark.parametrize("d,dtype", [(64, FP), (128, BF)])
def test_window_lengths(d, dtype, N):
    q, k, v = window_inputs(1, 2, 1, N, d, dtype, seed=N)
    check_window(q, k, v, 100, 4)
    check_window(q, k, v, 1, 0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 1), (2, 129), (64, 0), (127, 1), (128, 128), (129, 64), (300, 200),
                                          (1, 2 ** 31 - 1), (2 ** 31 - 1, 7), (640, 3)])
@pytest.mark.parametrize("d,dtype,layout", [(64, BF, "NHD"), (128, FP, "HND")])
def test_window_masks(d, dtype, layout, window, sinks):
    q, k, v = window_inputs(2, 4, 2, 700, d, dtype, seed=window % 1000)
    check_window(q, k, v, window, sinks, layout=layout)


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("d,dtype", [(64, FP), (64, BF), (128, FP), (128, BF)])
def test_window_padded_batches(d, dtype, layout):
    """Rows behind a sequence's end hold NaN, are not read and not written."""
    q, k, v = window_inputs(6, 3, 3, 391, d, dtype)
    check_window(q, k, v, 120, 5, lens=[0, 1, 128, 130, 391, 257], layout=layout)
    check_window(q, k, v, 0, 0, lens=[391, 0, 64, 3, 200, 390], layout=layout)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (12, 3), (8, 8)])
def test_window_head_groups_and_scale(Hq, Hkv):
    q, k, v = window_inputs(2, Hq, Hkv, 300, 64, BF)
    check_window(q, k, v, 70, 2, scale=0.4)


def test_window_growing_scores():
    """Keys whose scores grow along the sequence by far more than fp32's range of exponentials: the running
    maximum moves at every tile, and the first rows' sums must not be lost."""
    q, k, v = window_inputs(1, 2, 2, 600, 64, BF)
    q[:] = q.abs()
    k[:] = (k.float().abs() * torch.linspace(0.01, 6.0, 600)[:, None]).to(BF)
    check_window(q, k, v, 400, 4)
    check_window(q, k.flip(2), v, 400, 4)


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("what", ["k", "v"])
def test_window_values_of_unseen_keys_do_not_matter(what, bad):
    """A NaN or infinity in key or value j reaches the rows that see j (as NaN or infinity) and no other."""
    q, k, v = window_inputs(1, 2, 1, 300, 64, FP)
    ref, rl, to, tl = window_ref(q, k, v, 50, 2)
    for j in (100, 170, 290):
        (k if what == "k" else v)[0, 0, j, 7] = bad
    o, lse = sage.sage_attn_window_fwd_lse(q.cuda(), k.cuda(), v.cuda(), window=50, sinks=2)
    i = torch.arange(300)
    clean = ~(((i >= 100) & (i < 150)) | ((i >= 170) & (i < 220)) | (i >= 290))
    assert_within(o[:, :, clean], ref[:, :, clean], to[:, :, clean])
    assert_within(lse[:, :, clean], rl[:, :, clean], tl[:, :, clean])
    if what == "v":
        assert not torch.isfinite(o[:, :, ~clean][..., 7]).any()
        keep = [c for c in range(64) if c != 7]
        assert_within(o[:, :, ~clean][..., keep], ref[:, :, ~clean][..., keep], to[:, :, ~clean][..., keep])


def test_window_matches_decode_and_graph():
    """The last row of the prefill is the token that the decode attends with; a captured call replays."""
    N, window, sinks = 345, 100, 4
    q, k, v = (x.cuda() for x in window_inputs(2, 4, 2, N, 128, BF))
    o = sage.sage_attn_window_fwd(q, k, v, window=window, sinks=sinks)
    cache = sage.KVCache.alloc(60, 16, 2, 128, BF)
    table = torch.arange(44, dtype=torch.int32, device="cuda").view(2, 22)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    sage.sage_kv_append(k, v, cache, table, lens)
    one = sage.sage_attn_decode(q[:, :, -1].contiguous(), cache, table, lens + N, window=window, sinks=sinks)
    assert (one.float() - o[:, :, -1].float()).abs().max() <= 2 ** -6 * v.float().abs().max()
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sage.sage_attn_window_fwd(q, k, v, window=window, sinks=sinks, out=out)
    q2 = q.clone()
    q.copy_(q.flip(0))
    g.replay()
    torch.cuda.synchronize()
    want = sage.sage_attn_window_fwd(q2.flip(0).contiguous(), k, v, window=window, sinks=sinks)
    assert torch.equal(bits(out), bits(want))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("quantized,layout,dtype", [(False, "HND", BF), (True, "NHD", FP), (True, "HND", BF)])
def test_a_run_of_them_together(quantized, layout, dtype):
    """A padded batch of prompts through a local layer, its keys into the cache, new tokens with weights
    gathered, eviction, and more tokens: each step against the plain forms on what the cache then holds."""
    B, Hq, H, N, d, page, keep = 3, 4, 2, 200, 64, 16, 96
    lens = [200, 37, 150]
    q, k, v = window_inputs(B, Hq, H, N, d, dtype)
    check_window(q, k, v, 64, 4, lens=lens, layout=layout)
    c = Paged([0] * B, H, d, dtype, page, quantized=quantized, layout=layout, extra=240, weights=True,
              spare=3 + B * 8)
    cache, table, dl = c.to_gpu()

    def tokens(x):
        return (x if layout == "HND" else x.transpose(1, 2)).contiguous().cuda()

    n_new = torch.tensor(lens, dtype=torch.int32).cuda()
    sage.sage_kv_append(tokens(k), tokens(v), cache, table, dl, n_new=n_new, tensor_layout=layout)
    dl += n_new
    for b, n in enumerate(lens):
        c.put(b, 0, k[b, :, :n], v[b, :, :n])
    c.lens = list(lens)
    weight = torch.zeros((B, H, 240), dtype=torch.float64)
    g = torch.Generator().manual_seed(9)

    def step():
        kn, vn, qn = (torch.randn((B, X, 1, d), generator=g).to(dtype) for X in (H, H, Hq))
        sage.sage_kv_append(tokens(kn), tokens(vn), cache, table, dl, tensor_layout=layout)
        dl.add_(1)
        for b in range(B):
            c.put(b, c.lens[b], kn[b], vn[b])
            c.lens[b] += 1
        o, lse, to, tl, grown, err = decode_ref(c, qn[:, :, 0])
        got, got_lse = sage.sage_attn_decode_lse(qn[:, :, 0].contiguous().cuda(), cache, table, dl)
        assert_within(got, o, to)
        assert_within(got_lse, lse, tl)
        for b, (at, p) in enumerate(grown):
            weight[b][:, at] += p
        return err

    err = sum(step() for _ in range(5))
    used = [-(-n // page) for n in c.lens]
    w = cache.weight.cpu()
    for b in range(B):
        have = torch.cat([w[int(c.table[b, x])] for x in range(used[b])], 1)[:, :c.lens[b]].double()
        assert_within(have, weight[b][:, :c.lens[b]], (2.1 * err + 2.0 ** -17) * weight[b][:, :c.lens[b]] + 1e-6)
    dst = torch.full((B, 15), -1, dtype=torch.int32)
    dst[:, :8] = c.free[:B * 8].view(B, 8)
    dst = dst.cuda()
    new_lens, kept = sage.sage_kv_evict(cache, table, dl, dst, keep, sinks=4, recent=16)
    kept = kept.cpu()
    for b in range(B):
        for h in range(H):
            have = [w[c.slot(b, j)[0], h, c.slot(b, j)[1]] for j in range(c.lens[b])]
            stay = evict_ref(have, c.lens[b], keep, 4, 16)
            assert kept[b, h, :len(stay)].tolist() == stay
        at = kept[b, :, :min(keep, c.lens[b])].long()[..., None].expand(-1, -1, d)
        c.keys[b], c.values[b] = torch.gather(c.keys[b], 1, at), torch.gather(c.values[b], 1, at)
    c.lens = new_lens.tolist()
    weight.zero_()
    table, dl, c.table = dst, new_lens, dst.cpu()
    for _ in range(3):
        step()
