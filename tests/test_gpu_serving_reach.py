"""Ways through the serving kernels that take more heads, more items or more
replays than the tests of their masks: groups of heads in the sliding-window
kernel, joins of many heads, wide groups over long rows, weights gathered by
replayed graphs."""
import math

import pytest
import torch

from quantized_attention_block_b200 import sage

from serving_ref import Paged, assert_within, decode_ref, window_ref
from test_gpu_serving import bits, check_decode, no_device_error, window_inputs  # noqa: F401
from test_gpu_serving_edges import many_items, some_rows
from test_window_again import order

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("H,Hkv,d,window", [(11, 11, 128, 100), (11, 11, 128, 0), (22, 22, 64, 3000), (21, 21, 64, 3000)])
def test_window_groups_of_heads(H, Hkv, d, window):
    """Two groups of heads, the last one shorter for odd numbers: each head as it is in a call of its own, which has one group."""
    N = 8192
    items, group = order(1, H, Hkv, N, d)
    assert group < H
    q, k, v = many_items(N, d, BF, H, Hkv)
    o, lse = sage.sage_attn_window_fwd_lse(q, k, v, window=window, sinks=3)
    for h in range(H):
        one, one_lse = sage.sage_attn_window_fwd_lse(*(x[:, h:h + 1].contiguous() for x in (q, k, v)), window=window,
                                                     sinks=3)
        assert torch.equal(bits(o[:, h]), bits(one[:, 0])) and torch.equal(lse[:, h], one_lse[:, 0])
    rows = torch.tensor([0, 255, 256, 5000, 8191])
    for h in (0, group - 1, group, H - 1):
        ref, tol = some_rows(q, k, v, 0, h, rows, window, 3)
        assert_within(o[0, h, rows], ref, tol)


@pytest.mark.parametrize("lens", [[700, 0, 1, 530, 900], [600, 850]])
@pytest.mark.parametrize("d,quantized", [(128, False), (64, True)])
def test_decode_joins_of_many_heads_and_of_few(lens, d, quantized):
    """320 heads (joined by 128 threads each) and 128 (by 512), over split rows."""
    check_decode(Paged(lens, 8, d, BF, 16, quantized=quantized, weights=True), 64)


@pytest.mark.parametrize("G", [9, 16, 17, 33])
@pytest.mark.parametrize("d,dtype,layout", [(128, BF, "HND"), (64, FP, "NHD"), (128, FP, "NHD")])
def test_decode_wide_groups_over_split_rows(d, dtype, layout, G):
    check_decode(Paged([700, 300, 0, 1100], 3, d, dtype, 32, layout=layout, weights=G in (16, 17)), 3 * G)


@pytest.mark.parametrize("longest,window", [(400, 0), (900, 0), (900, 64)])
def test_replayed_graphs_gather_weights(longest, window):
    """A captured decode with weights, replayed with other lengths: outputs and weights of every replay."""
    c = Paged([longest, 33, 350], 2, 128, BF, 16, weights=True)
    cache, table, lens = c.to_gpu()
    g = torch.Generator().manual_seed(4)
    q = torch.randn((3, 8, 128), generator=g).to(BF)
    qd, out = q.cuda(), torch.empty((3, 8, 128), dtype=BF, device="cuda")
    ws = torch.empty(sage.decode_workspace_bytes(cache, table, lens, 8, window=window, sinks=2), dtype=torch.uint8,
                     device="cuda")
    before = cache.weight.clone()
    sage.sage_attn_decode(qd, cache, table, lens, window=window, sinks=2, out=out, workspace=ws)
    torch.cuda.synchronize()
    cache.weight.copy_(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sage.sage_attn_decode(qd, cache, table, lens, window=window, sinks=2, out=out, workspace=ws)
    want, tol = c.weight.double().clone(), torch.zeros(c.weight.shape, dtype=torch.float64)
    for new in ([longest, 33, 350], [1, 0, 77], [longest - 1, 32, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        c.lens = new
        o, _, to, _, grown, err = decode_ref(c, q, window, 2)
        assert_within(out, o, to)
        for b, at_p in enumerate(grown):
            for j, p in zip(at_p[0].tolist(), at_p[1].T) if at_p else ():
                pid, r = c.slot(b, j)
                want[pid, :, r] += p
                # as in check_decode, a replay after the other
                tol[pid, :, r] += (2.1 * err + 2.0 ** -19) * p + 4 * 2.0 ** -23 * want[pid, :, r].abs()
        assert_within(cache.weight, want, tol)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 2), (70, 3), (130, 64), (200, 130), (64, 65), (500, 1)])
@pytest.mark.parametrize("d,dtype,layout", [(64, FP, "NHD"), (128, BF, "HND"), (128, FP, "NHD")])
def test_window_bad_values_in_many_places(d, dtype, layout, window, sinks):
    """NaN and infinities at random in V: a channel of a row is not finite if the row sees one there, and what it would
    be without them else; padded batches, grouped heads."""
    B, Hq, Hkv, N, lens = 3, 4, 2, 700, [700, 0, 431]
    q, k, v = window_inputs(B, Hq, Hkv, N, d, dtype, seed=window)
    ref, rl, to, tl = window_ref(q, k, v, window, sinks, lens)
    g = torch.Generator().manual_seed(sinks)
    bad = torch.zeros(v.shape, dtype=torch.bool)
    for _ in range(12):
        b, h, j, c = (int(torch.randint(0, n, (1,), generator=g)) for n in (B, Hkv, N, d))
        bad[b, h, j, c] = True
        v[b, h, j, c] = (math.nan, math.inf, -math.inf)[j % 3]
    for b, n in enumerate(lens):
        for x in (q, k, v):
            x[b, :, n:] = math.nan
        bad[b, :, n:] = False
    x = [(t if layout == "HND" else t.transpose(1, 2)).contiguous().cuda() for t in (q, k, v)]
    o, lse = sage.sage_attn_window_fwd_lse(*x, window=window, sinks=sinks, lens=torch.tensor(lens).int().cuda(),
                                           tensor_layout=layout)
    o = (o if layout == "HND" else o.transpose(1, 2)).cpu()
    p, j = torch.arange(N)[:, None], torch.arange(N)[None]
    see = (j <= p) & ((p - j < window) | (j < sinks) | (window == 0))
    hit = (see.double() @ bad.double() > 0).repeat_interleave(Hq // Hkv, 1)
    live = ~torch.isnan(ref)
    assert not torch.isfinite(o[hit & live]).any()
    assert_within(o[~hit & live], ref[~hit & live], to[~hit & live], "o")
    assert (o[~live] == 0).all()
    rows = ~torch.isnan(rl)
    assert_within(lse.cpu()[rows], rl[rows], tl[rows], "lse")
