"""Plain 64-bit forms of the serving operators (paged cache, one-token and
sliding-window attention, eviction) on the CPU, and their error bounds."""
from __future__ import annotations

import math

import torch

from quantized_attention_block_b200 import sage

NAN = float("nan")
# one rounding to the output's type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def visible(p: int, n: int, window: int, sinks: int) -> torch.Tensor:
    """Positions that a query at p sees among n keys."""
    j = torch.arange(min(n, p + 1))
    return j if window == 0 else j[(p - j < window) | (j < sinks)]


def score_error(q, k, scale: float) -> float:
    """Bound of a score's error: every product of two 16-bit (or INT8) numbers is exact in fp32; the d products
    are added in at most d / 16 + 4 roundings (or truncations, twice as large) of partial sums below
    sum |q| |k|; the scaling adds two roundings."""
    a = (q.abs().double() @ k.abs().double().transpose(-1, -2)).max().item() * scale if k.numel() else 0.0
    return (q.shape[-1] / 16 + 6) * 2.0 ** -23 * a


def softmax_rows(q, k, v, scale):
    """o, lse, p of rows q [.., m, d] over keys k [.., n, d] in 64 bits."""
    t = (q.double() @ k.double().transpose(-1, -2)) * scale
    z = torch.logsumexp(t, -1, keepdim=True)
    p = torch.exp(t - z)
    return p @ v.double(), z[..., 0], p


def out_tol(ref, v, err: float, dtype) -> torch.Tensor:
    """|o - ref|: the output's rounding; scores off by err move the weights by a factor e^(+-2 err), which moves o by
    at most 4 err max|v|; 2^-15 for the weights' two 16-bit parts, the exponentials and the sums in fp32."""
    vmax = v.abs().max().item() if v.numel() else 0.0
    return HALF_STEP[dtype] * ref.abs() + (4 * err + 2.0 ** -15) * vmax + 1e-30


def quantize(k, v, km=None):
    """INT8 keys and E4M3 values with a scale per row, as sage_kv_append defines them (fp32)."""
    x = k.float() if km is None else k.float() - km
    ks = x.abs().amax(-1) / torch.tensor(127.0)
    vs = v.float().abs().amax(-1) / torch.tensor(448.0)
    one = torch.ones(())
    kc = torch.clamp(torch.round(x / torch.where(ks > 0, ks, one)[..., None]), -127, 127)
    vc = v.float() / torch.where(vs > 0, vs, one)[..., None]
    return kc.to(torch.int8), vc.to(torch.float8_e4m3fn), ks, vs


class Paged:
    """A cache on the host with every slot that holds no token NaN (scales too), pages in random order, and
    page-table entries behind a sequence's pages out of range."""

    def __init__(self, lens, Hkv, d, dtype, page, *, quantized=False, layout="HND", seed=0, spare=3, extra=0,
                 weights=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.d, self.dtype, self.page = list(lens), Hkv, d, dtype, page
        self.quantized, self.layout = quantized, layout
        used = [-(-(n + extra) // page) for n in lens]
        self.n_pages = sum(used) + spare
        perm = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.max_pages = max(1, max(used))
        self.table = torch.full((len(lens), self.max_pages), -12345, dtype=torch.int32)
        self.table[::2] = 2 ** 30
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = perm[at:at + u]
            at += u
        self.free = perm[at:]
        shape = (self.n_pages, Hkv, page, d)
        self.k, self.v = torch.full(shape, NAN, dtype=dtype), torch.full(shape, NAN, dtype=dtype)
        self.ks = torch.full(shape[:3], NAN)
        self.vs = torch.full(shape[:3], NAN)
        self.kc = torch.full(shape, 77, dtype=torch.int8)
        self.vc = torch.full(shape, 0x7F, dtype=torch.int8).view(torch.float8_e4m3fn)
        self.weight = torch.rand(shape[:3], generator=g) * 3 if weights else None
        self.keys, self.values = [], []  # [Hkv, n, d] as the cache holds them, in 64 bits
        bias = 2.0 * torch.randn((Hkv, 1, d), generator=g)
        for b, n in enumerate(lens):
            k = (torch.randn((Hkv, n, d), generator=g) + bias).to(dtype)
            v = torch.randn((Hkv, n, d), generator=g).to(dtype)
            self.put(b, 0, k, v)

    def slot(self, b, pos):
        return int(self.table[b, pos // self.page]), pos % self.page

    def put(self, b, pos, k, v):
        kc, vc, ks, vs = quantize(k, v)
        for i in range(k.shape[1]):
            pid, r = self.slot(b, pos + i)
            self.k[pid, :, r], self.v[pid, :, r] = k[:, i], v[:, i]
            self.kc[pid, :, r], self.ks[pid, :, r], self.vs[pid, :, r] = kc[:, i], ks[:, i], vs[:, i]
            self.vc.view(torch.int8)[pid, :, r] = vc.view(torch.int8)[:, i]
        if self.quantized:
            k, v = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
        if b == len(self.keys):
            self.keys.append(k.double())
            self.values.append(v.double())
        else:
            self.keys[b] = torch.cat([self.keys[b], k.double()], 1)
            self.values[b] = torch.cat([self.values[b], v.double()], 1)

    def hide(self, b, positions):
        """NaN in tokens that a call must not look at."""
        for pos in positions:
            pid, r = self.slot(b, int(pos))
            self.k[pid, :, r] = self.v[pid, :, r] = NAN
            self.ks[pid, :, r] = self.vs[pid, :, r] = NAN

    def to_gpu(self):
        def lay(x):
            return (x if self.layout == "HND" else x.transpose(1, 2)).contiguous().cuda()

        if self.quantized:
            vc = lay(self.vc.view(torch.int8)).view(torch.float8_e4m3fn)
            c = sage.KVCache(lay(self.kc), vc, self.ks.cuda(), self.vs.cuda(),
                             None if self.weight is None else self.weight.cuda(), tensor_layout=self.layout)
        else:
            c = sage.KVCache(lay(self.k), lay(self.v), weight=None if self.weight is None else self.weight.cuda(),
                             tensor_layout=self.layout)
        return c, self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()


def decode_ref(cache: Paged, q, window=0, sinks=0, scale=None):
    """(o, lse, tolerance of o, of lse, [p of each sequence: Hkv, n_visible], score error) in 64 bits."""
    B, Hq, d = q.shape
    G = Hq // cache.Hkv
    scale = scale or 1.0 / math.sqrt(d)
    o, lse = torch.zeros((B, Hq, d), dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    grown, worst = [], 0.0
    for b, n in enumerate(cache.lens):
        if n == 0:
            grown.append(None)
            continue
        at = visible(n - 1, n, window, sinks)
        k, v = cache.keys[b][:, at], cache.values[b][:, at]
        qq = q[b].double().view(cache.Hkv, G, d)
        ob, zb, p = softmax_rows(qq, k, v, scale)
        err = score_error(qq, k, scale)
        worst = max(worst, err)
        o[b], lse[b] = ob.reshape(Hq, d), zb.reshape(Hq)
        to[b] = out_tol(o[b], v, err, q.dtype)
        tl[b] = err + 2.0 ** -21 * (4 + lse[b].abs())
        grown.append((at, p.sum(1)))
    return o, lse, to, tl, grown, worst


def assert_within(got, ref, tol, what=""):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol) & ~((got == ref))
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: "
                             f"{got[at].item()} against {ref[at].item()}, tolerance {tol[at].item()}")


def window_ref(q, k, v, window, sinks, lens=None, scale=None):
    """(o, lse, tolerances) of HND tensors in 64 bits; rows behind lens hold NaN."""
    B, Hq, N, d = q.shape
    G = Hq // k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    o, lse = torch.full((B, Hq, N, d), NAN, dtype=torch.float64), torch.full((B, Hq, N), NAN, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = N if lens is None else lens[b]
        if n == 0:
            continue
        p, j = torch.arange(n)[:, None], torch.arange(n)[None]
        hidden = (j > p) | ((p - j >= window) & (j >= sinks)) if window else j > p
        for h in range(Hq):
            kk, vv = k[b, h // G, :n].double(), v[b, h // G, :n].double()
            t = (q[b, h, :n].double() @ kk.T) * scale
            t[hidden] = -math.inf
            z = torch.logsumexp(t, -1, keepdim=True)
            w = torch.exp(t - z)
            o[b, h, :n], lse[b, h, :n] = w @ vv, z[:, 0]
            err = score_error(q[b, h, :n], kk, scale)
            # the weights enter the tensor cores in the inputs' type: each off by half a step, relative, and
            # their sum (taken before that rounding) as much again
            to[b, h, :n] = out_tol(o[b, h, :n], vv, err, q.dtype) + 2 * HALF_STEP[q.dtype] * (w @ vv.abs())
            tl[b, h, :n] = err + 2.0 ** -21 * (4 + lse[b, h, :n].abs())
    return o, lse, to, tl


def evict_ref(weight, n, keep, sinks, recent):
    """Positions that stay of one head, in order."""
    if n <= keep:
        return list(range(n))
    cand = range(sinks, n - recent)

    def rank(j):
        w = float(weight[j])
        return (1, 0.0, j) if math.isnan(w) else (0, -w, j)

    top = sorted(cand, key=rank)[:keep - sinks - recent]
    return list(range(sinks)) + sorted(top) + list(range(n - recent, n))
