"""Workloads of the serving operators: the paged key-value cache (append,
attention of a new token, eviction) and sliding-window attention with sinks.

Each case is one call of one operator.  `own` chooses what `run` calls: the
library's entry points, or the operators' plain forms in elementary torch
operations (32-bit arithmetic, one rounding at the end).  `exact` states the
operators once more in 64 bits.

Visibility, for a query at position p and a key at j < length:
    j <= p and (window == 0 or p - j < window or j < sinks)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step's new tokens of 64 short chats into an 8-bit cache: launch latency
        dict(name="append_step_b64_8bit", op="append", B=64, Hkv=8, d=128, T=1, dtype="bf16", cache="8", page=16,
             layout="HND", held=200),
        # eight ragged prompts, as a prefill leaves them, into a 16-bit cache: pure bandwidth
        dict(name="append_prompts_b8_t4096", op="append", B=8, Hkv=8, d=128, T=4096, dtype="bf16", cache="16",
             page=64, layout="HND", held=0),
        # the first answers to one short question: the smallest call, latency counts
        dict(name="decode_one_len201", op="decode", B=1, Hq=32, Hkv=8, d=128, dtype="bf16", cache="16", page=16,
             layout="HND", shortest=201, longest=201, window=0, sinks=0, track=False),
        # a serving batch of ragged lengths, grouped heads
        dict(name="decode_b32_ragged8k", op="decode", B=32, Hq=32, Hkv=8, d=128, dtype="bf16", cache="16", page=16,
             layout="HND", shortest=513, longest=8191, window=0, sinks=0, track=False),
        # one long document, 8-bit cache: few rows, split over a long axis
        dict(name="decode_b1_131k_8bit", op="decode", B=1, Hq=32, Hkv=8, d=128, dtype="bf16", cache="8", page=64,
             layout="HND", shortest=131001, longest=131001, window=0, sinks=0, track=False),
        # a local layer's step (window and sinks) of 16 long chats, ungrouped heads, weights accumulated
        dict(name="decode_window_track_fp16", op="decode", B=16, Hq=24, Hkv=24, d=64, dtype="fp16", cache="16",
             page=32, layout="NHD", shortest=777, longest=16001, window=1024, sinks=4, track=True),
        # the largest step: 64 chats of up to 12k tokens, 64 query heads
        dict(name="decode_b64_ragged12k", op="decode", B=64, Hq=64, Hkv=8, d=128, dtype="bf16", cache="16", page=64,
             layout="HND", shortest=1024, longest=12288, window=0, sinks=0, track=False),
        # a padded batch of short prompts through a local layer: latency
        dict(name="window_short_padded_fp16", op="window", B=3, Hq=4, Hkv=2, N=333, d=64, dtype="fp16", window=100,
             sinks=4, layout="NHD", padded=True),
        # a local layer of the prefill recipe: B4 H32 N4096 d128
        dict(name="window_b4_h32_n4096", op="window", B=4, Hq=32, Hkv=32, N=4096, d=128, dtype="bf16", window=1024,
             sinks=4, layout="HND", padded=False),
        # a long grouped-head prompt with a wide window
        dict(name="window_gqa_n8192", op="window", B=1, Hq=32, Hkv=8, N=8192, d=128, dtype="bf16", window=4096,
             sinks=16, layout="HND", padded=False),
        # four short chats held to a small budget
        dict(name="evict_b4_to512", op="evict", B=4, Hkv=8, d=128, dtype="bf16", cache="16", page=16, layout="HND",
             shortest=300, longest=1200, keep=512, sinks=4, recent=64),
        # sixteen long chats halved, 8-bit cache
        dict(name="evict_b16_to12k_8bit", op="evict", B=16, Hkv=8, d=128, dtype="bf16", cache="8", page=64,
             layout="HND", shortest=10001, longest=32768, keep=12288, sinks=16, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "window", "window", "evict"])
    c = dict(op=op, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]), layout=rng.choice(["HND", "NHD"]))
    if op != "window":
        c.update(cache=rng.choice(["16", "8"]), page=rng.choice([16, 32, 64, 128]), Hkv=rng.choice([1, 2, 4, 5, 8, 16]))
    if op == "append":
        c["B"] = _log_int(rng, 1, 64)
        c["T"] = _log_int(rng, 1, max(1, min(4096, (1 << 18) // (c["B"] * c["Hkv"]))))
        c["held"] = _log_int(rng, 1, 4000) - 1
    elif op == "decode":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 6, 8, 12, 16] if c["Hkv"] <= 4 else [1, 2, 4, 6, 8])
        c["B"] = _log_int(rng, 1, 64)
        c["longest"] = _log_int(rng, 1, max(1, min(131072, 3000000 // (c["B"] * c["Hkv"]))))
        c["shortest"] = rng.choice([0, 1, max(1, c["longest"] // 7), c["longest"]])
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        c["sinks"] = rng.choice([0, 1, 4, 33]) if c["window"] else 0
        c["track"] = rng.random() < 0.3
    elif op == "window":
        c["Hkv"] = rng.choice([1, 2, 4, 8])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4])
        c["B"] = rng.choice([1, 2, 3])
        most = int(math.sqrt(1.0e9 / (c["B"] * c["Hq"])))
        c["N"] = _log_int(rng, 1, min(8192, most))
        c["window"] = _log_int(rng, 1, max(1, c["N"]))
        c["sinks"] = rng.choice([0, 1, 4, 16, 130])
        c["padded"] = rng.random() < 0.5
    else:
        c["B"] = _log_int(rng, 1, 16)
        c["longest"] = _log_int(rng, 16, min(32768, 2000000 // (c["B"] * c["Hkv"])))
        c["shortest"] = rng.choice([0, max(1, c["longest"] // 5), c["longest"]])
        c["keep"] = max(1, int(c["longest"] * rng.uniform(0.2, 0.9)))
        c["sinks"] = min(rng.choice([0, 4, 16]), c["keep"] // 4)
        c["recent"] = int((c["keep"] - c["sinks"]) * rng.choice([0.0, 0.1, 0.5]))
    return c


def _lengths(B, shortest, longest):
    """B lengths from shortest to longest (evenly spread, both ends included)."""
    return [longest] if B == 1 else [shortest + (longest - shortest) * b // (B - 1) for b in range(B)]


def _new_tokens(c):
    """Tokens that each sequence appends: T for one-token steps, else ragged up to T."""
    return [max(1, c["T"] * (b + 1) // c["B"]) for b in range(c["B"])]


def _visible(n, window, sinks):
    """Keys that the query at position n - 1 sees."""
    return n if window == 0 or n <= window else window + min(sinks, n - window)


# ---------------------------------------------------------------- inputs
def _row_scale(x, top):
    """max |x| over the channels, divided by `top` (a tensor, so that the division is a division)."""
    return x.abs().amax(-1) / torch.full((), top, dtype=x.dtype, device=x.device)


def _code(x, s):
    return torch.where(s[..., None] > 0, x / torch.where(s > 0, s, torch.ones_like(s))[..., None], torch.zeros_like(x))


def _pools(c, n_pages, g, km, like_real):
    """Key and value pages [n_pages, Hkv, page, d] (HND) or [n_pages, page, Hkv, d] (NHD), with scales for 8 bits."""
    H, P, d = c["Hkv"], c["page"], c["d"]
    shape = (n_pages, H, P, d) if c["layout"] == "HND" else (n_pages, P, H, d)
    dt = DTYPES[c["dtype"]]
    if not like_real:
        k, v = torch.zeros(shape, dtype=dt, device="cuda"), torch.zeros(shape, dtype=dt, device="cuda")
    else:
        k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        if c["cache"] == "16":  # keys share a bias a channel, as the prefill recipes have it
            k += km.to(dt).mean(0)[:, None, :] if c["layout"] == "HND" else km.to(dt).mean(0)
    if c["cache"] == "16":
        return k, v, None, None
    ks, vs = _row_scale(k.float(), 127.0), _row_scale(v.float(), 448.0)
    k8 = torch.clamp(torch.round(_code(k.float(), ks)), -127, 127).to(torch.int8)
    v8 = _code(v.float(), vs).to(torch.float8_e4m3fn)
    if c["layout"] == "NHD":
        ks, vs = ks.transpose(1, 2), vs.transpose(1, 2)
    return k8, v8, ks.contiguous(), vs.contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def heads(B, H, N, d):
        return randn(B, H, N, d).to(dt) if c["layout"] == "HND" else randn(B, N, H, d).to(dt)

    s = dict(case=c)
    B, d = c["B"], c["d"]
    order = torch.randperm(B, generator=g, device="cuda")
    if c["op"] == "window":
        s["q"], s["k"], s["v"] = heads(B, c["Hq"], c["N"], d), heads(B, c["Hkv"], c["N"], d), heads(B, c["Hkv"], c["N"], d)
        bias = 3.0 * randn(1, c["Hkv"], 1, d)
        s["k"] += (bias if c["layout"] == "HND" else bias.transpose(1, 2)).to(dt)
        s["lens"] = None
        if c["padded"]:
            s["lens"] = torch.tensor(_lengths(B, c["N"] // 2, c["N"]), dtype=torch.int32, device="cuda")[order]
        return s

    # pages of the sequences, in no order, out of a pool with a few pages to spare
    if c["op"] == "append":
        n_new, held = _new_tokens(c), [c["held"] * (b + 1) // B for b in range(B)]
        longest = max(n + h for n, h in zip(n_new, held))
        s["n_new"] = torch.tensor(n_new, dtype=torch.int32, device="cuda")[order]
        s["lens"] = torch.tensor(held, dtype=torch.int32, device="cuda")[order]
    else:
        lens = _lengths(B, c["shortest"], c["longest"])
        longest = max(lens)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
    per = max(1, -(-longest // c["page"]))
    dst_per = -(-c["keep"] // c["page"]) if c["op"] == "evict" else 0
    n_pages = B * (per + dst_per) + 3
    pages = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = pages[:B * per].view(B, per)
    s["dst_table"] = pages[B * per:B * (per + dst_per)].view(B, dst_per)
    s["km"] = 3.0 * randn(B, c["Hkv"], d) if c["cache"] == "8" else None
    s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"] = _pools(
        c, n_pages, g, 3.0 * randn(B, c["Hkv"], d), c["op"] != "append")
    s["weight"] = None
    if c["op"] == "evict" or c.get("track"):  # attention weight gathered so far: a few heavy keys, many light ones
        s["weight"] = torch.exp(2.0 * randn(n_pages, c["Hkv"], c["page"]))
    if c["op"] == "append":
        s["k"], s["v"] = heads(B, c["Hkv"], c["T"], d), heads(B, c["Hkv"], c["T"], d)
        if c["cache"] == "8":
            bias = s["km"][:, :, None] if c["layout"] == "HND" else s["km"][:, None]
            s["k"] = (s["k"].float() + bias).to(dt)
    elif c["op"] == "decode":
        s["q"] = randn(B, c["Hq"], d).to(dt)
    if own:  # the handle that a serving program keeps with its pages
        from quantized_attention_block_b200 import sage
        s["cache"] = sage.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["weight"],
                                  tensor_layout=c["layout"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from quantized_attention_block_b200 import sage
    c = s["case"]
    if c["op"] == "append":
        sage.sage_kv_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], n_new=s["n_new"], km=s["km"],
                            tensor_layout=c["layout"])
        return _state_of(s)
    if c["op"] == "decode":
        o, lse = sage.sage_attn_decode_lse(s["q"], s["cache"], s["table"], s["lens"], window=c["window"],
                                           sinks=c["sinks"], km=s["km"])
        return [o, lse] + ([s["weight"]] if c["track"] else [])
    if c["op"] == "window":
        return list(sage.sage_attn_window_fwd_lse(s["q"], s["k"], s["v"], window=c["window"], sinks=c["sinks"],
                                                  lens=s["lens"], tensor_layout=c["layout"]))
    new_lens, kept = sage.sage_kv_evict(s["cache"], s["table"], s["lens"], s["dst_table"], c["keep"],
                                        sinks=c["sinks"], recent=c["recent"])
    return [new_lens, kept, s["weight"]] + _state_of(s)


def _state_of(s):
    return [s["k_pages"], s["v_pages"]] + ([s["k_scale"], s["v_scale"]] if s["k_scale"] is not None else [])


def _run_plain(s):
    return {"append": _plain_append, "decode": _plain_decode, "window": _plain_window,
            "evict": _plain_evict}[s["case"]["op"]](s)


def _slots(table, page, positions):
    """(page id, row) of the positions [B, n]."""
    p = torch.clamp(positions.long(), 0, table.shape[1] * page - 1)
    return torch.gather(table.long(), 1, p // page), p % page


def _put(pool, layout, ids, rows, values, where):
    """pool[ids[b, n], :, rows[b, n]] = values[b, :, n] where `where`[b, n]."""
    b, n = torch.nonzero(where, as_tuple=True)
    x = values.transpose(1, 2)[b, n]  # [m, H, ...]
    if layout == "HND":
        pool.transpose(1, 2)[ids[b, n], rows[b, n]] = x
    else:
        pool[ids[b, n], rows[b, n]] = x


def _plain_append(s):
    c = s["case"]
    k, v = (x if c["layout"] == "HND" else x.transpose(1, 2) for x in (s["k"], s["v"]))
    t = torch.arange(c["T"], device=k.device)
    ids, rows = _slots(s["table"], c["page"], s["lens"][:, None] + t)
    new = t[None] < s["n_new"][:, None]
    if c["cache"] == "8":
        x, v = k.float() - s["km"][:, :, None], v.float()
        ks, vs = _row_scale(x, 127.0), _row_scale(v, 448.0)
        k = torch.clamp(torch.round(_code(x, ks)), -127, 127).to(torch.int8)
        v = _code(v, vs).to(torch.float8_e4m3fn).view(torch.int8)
        _put(s["k_scale"], "HND", ids, rows, ks, new)
        _put(s["v_scale"], "HND", ids, rows, vs, new)
        _put(s["v_pages"].view(torch.int8), c["layout"], ids, rows, v, new)
    else:
        _put(s["v_pages"], c["layout"], ids, rows, v, new)
    _put(s["k_pages"], c["layout"], ids, rows, k, new)
    return _state_of(s)


def _gathered(s, pool, scale=None, to=torch.float32):
    """A pool's pages of each sequence, in order: [B, Hkv, L, d], dequantised."""
    t = s["table"].long()
    x = (pool.view(torch.int8)[t].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[t]).to(to)
    x = x if s["case"]["layout"] == "HND" else x.transpose(2, 3)
    if scale is not None:
        x = x * scale[t].to(to)[..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_decode(s):
    c = s["case"]
    B, H, G, d = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    k = _gathered(s, s["k_pages"], s["k_scale"])
    v = _gathered(s, s["v_pages"], s["v_scale"])
    q = s["q"].float().view(B, H, G, d)
    j = torch.arange(k.shape[2], device=q.device)
    n = s["lens"].long()[:, None]
    see = j < n
    if c["window"]:
        see &= (n - 1 - j < c["window"]) | (j < c["sinks"])
    see = see[:, None, None]
    t = (q @ k.transpose(2, 3)) * d ** -0.5
    t = t.masked_fill_(~see, float("-inf"))
    m = t.amax(-1, keepdim=True)
    e = torch.exp(t - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, torch.ones_like(total), total)
    o = (p @ torch.where(see.squeeze(2)[..., None], v, torch.zeros_like(v))).view(B, H * G, d).to(s["q"].dtype)
    lse = (m + torch.log(total)).view(B, H, G)
    if s["km"] is not None:
        lse = lse + d ** -0.5 * (q * s["km"][:, :, None]).sum(-1)
    out = [o, lse.reshape(B, H * G)]
    if c["track"]:
        ids, rows = _slots(s["table"], c["page"], j[None].expand(B, -1))
        b, at = torch.nonzero(see[:, 0, 0], as_tuple=True)
        s["weight"].transpose(1, 2)[ids[b, at], rows[b, at]] += p.sum(2).transpose(1, 2)[b, at]
        out.append(s["weight"])
    return out


def _window_mask(c, device, lens):
    """[B or 1, 1, N, N] visibility."""
    i = torch.arange(c["N"], device=device)
    ago = i[:, None] - i[None]
    see = (ago >= 0) & ((ago < c["window"]) | (i[None] < c["sinks"]))
    return see[None, None] if lens is None else see[None, None] & (i[None, None, None] < lens[:, None, None, None])


def _plain_window(s):
    c = s["case"]
    B, H, G, N, d = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["N"], c["d"]
    q, k, v = (x if c["layout"] == "HND" else x.transpose(1, 2) for x in (s["q"], s["k"], s["v"]))
    q = q.float().reshape(B, H, G, N, d)
    see = _window_mask(c, q.device, s["lens"])[:, :, None]
    t = (q @ k.float().transpose(2, 3)[:, :, None]).mul_(d ** -0.5)
    t.masked_fill_(~see, float("-inf"))
    m = t.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    e = t.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e @ v.float()[:, :, None]) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(B, H * G, N, d).to(s["q"].dtype)
    lse = (m + torch.log(total)).view(B, H * G, N)
    if s["lens"] is not None:  # rows behind a sequence's end
        past = torch.arange(N, device=q.device)[None, None] >= s["lens"][:, None, None]
        o = o.masked_fill(past[..., None], 0.0)
        lse = lse.masked_fill(past, 0.0)
    return [o if c["layout"] == "HND" else o.transpose(1, 2).contiguous(), lse]


def _plain_evict(s):
    c = s["case"]
    page, keep = c["page"], c["keep"]
    w = s["weight"][s["table"].long()].transpose(1, 2).flatten(2, 3)  # [B, Hkv, L]
    w = torch.where(torch.isnan(w), torch.full_like(w, float("-inf")), w)
    B, H, L = w.shape
    j = torch.arange(L, device=w.device)
    n = s["lens"].long()[:, None]
    held = (j < n)[:, None].expand(B, H, L)
    cand = ((j >= c["sinks"]) & (j < n - c["recent"]))[:, None].expand(B, H, L)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1]
    order = torch.gather(order, -1, torch.sort((~torch.gather(cand, -1, order)).to(torch.int8), dim=-1, stable=True)[1])
    rank = torch.empty_like(order).scatter_(-1, order, j.expand(B, H, L).contiguous())
    stay = torch.where((n <= keep)[:, None], held, held & (~cand | (rank < keep - c["sinks"] - c["recent"])))
    new_lens = torch.clamp(s["lens"], max=keep)
    slot = torch.sort((~stay).to(torch.int8), dim=-1, stable=True)[1][..., :keep]
    slot = torch.nn.functional.pad(slot, (0, keep - slot.shape[-1]))
    i = torch.arange(keep, device=w.device)
    valid = i < new_lens[:, None]
    kept = torch.where(valid[:, None], slot, torch.full_like(slot, -1)).to(torch.int32)
    ids, rows = _slots(s["dst_table"], page, i[None].expand(B, -1))
    from_id = torch.gather(s["table"].long()[:, None].expand(-1, H, -1), 2, slot // page)
    h = torch.arange(H, device=w.device)[None, :, None]
    v_pages = s["v_pages"].view(torch.int8) if s["v_pages"].dtype == torch.float8_e4m3fn else s["v_pages"]
    where = (from_id, h, slot % page, ids, rows, valid)
    _move(s["k_pages"], c["layout"], *where)
    _move(v_pages, c["layout"], *where)
    _move(s["weight"], "HND", *where)
    if c["cache"] == "8":
        _move(s["k_scale"], "HND", *where)
        _move(s["v_scale"], "HND", *where)
    return [new_lens, kept, s["weight"]] + _state_of(s)


def _move(pool, layout, from_id, h, from_row, ids, rows, valid):
    x = pool[from_id, h, from_row] if layout == "HND" else pool[from_id, from_row, h]
    _put(pool, layout, ids, rows, x, valid)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "append":
        return _exact_append(s)
    if op == "decode":
        return _exact_decode(s)
    if op == "window":
        return _exact_window(s)
    return _exact_evict(s)


def _exact_append(s):
    c = s["case"]
    quant = c["cache"] == "8"
    out = [s["k_pages"].double() if not quant else None, s["v_pages"].double()]
    if quant:
        out += [s["k_scale"].double(), s["v_scale"].double()]
    table, lens, n_new = s["table"].tolist(), s["lens"].tolist(), s["n_new"].tolist()
    for b in range(c["B"]):
        i = 0
        while i < n_new[b]:
            pos = lens[b] + i
            m = min(n_new[b] - i, c["page"] - pos % c["page"])  # up to the end of the page
            pid, r = table[b][pos // c["page"]], pos % c["page"]
            k, v = (x[b, :, i:i + m] if c["layout"] == "HND" else x[b, i:i + m].transpose(0, 1)
                    for x in (s["k"], s["v"]))
            k, v = k.double(), v.double()
            if quant:
                # km and the difference from it are held in 32 bits by definition
                x = (k.float() - s["km"][b][:, None]).double()
                out[2][pid, :, r:r + m] = x.abs().amax(-1) / 127.0
                out[3][pid, :, r:r + m] = v.abs().amax(-1) / 448.0
                sv = out[3][pid, :, r:r + m, None]
                v = (v / torch.where(sv > 0, sv, torch.ones_like(sv))).float().to(torch.float8_e4m3fn).double()
            for at, x in ((0, k), (1, v)):
                if out[at] is not None and c["layout"] == "HND":
                    out[at][pid, :, r:r + m] = x
                elif out[at] is not None:
                    out[at][pid, r:r + m] = x.transpose(0, 1)
            i += m
    return out


def _exact_decode(s):
    c = s["case"]
    B, H, G, d = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    o = torch.zeros((B, c["Hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"]), float("-inf"), dtype=torch.float64, device="cuda")
    weight = s["weight"].double() if c["track"] else None
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        used = -(-n // c["page"])
        ids = s["table"][b, :used].long()

        def rows(pool, scale):
            x = (pool.view(torch.int8)[ids].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[ids])
            x = x.double() if c["layout"] == "HND" else x.double().transpose(1, 2)
            if scale is not None:
                x = x * scale[ids].double()[..., None]
            return x.transpose(0, 1).reshape(H, used * c["page"], d)[:, :n]

        k, v = rows(s["k_pages"], s["k_scale"]), rows(s["v_pages"], s["v_scale"])
        at = torch.arange(n, device="cuda")
        if c["window"] and n > c["window"]:
            at = torch.cat([at[:min(c["sinks"], n - c["window"])], at[n - c["window"]:]])
        k, v = k[:, at], v[:, at]
        q = s["q"][b].double().view(H, G, d)
        t = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(d)
        z = torch.logsumexp(t, -1, keepdim=True)
        p = torch.exp(t - z)
        o[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(H * G, d)
        z = z[..., 0]
        if s["km"] is not None:
            z = z + torch.einsum("hgd,hd->hg", q, s["km"][b].double()) / math.sqrt(d)
        lse[b] = z.reshape(H * G)
        if weight is not None:
            weight[s["table"][b].long()[at // c["page"]], :, at % c["page"]] += p.sum(1).transpose(0, 1)
    return [o, lse] + ([weight] if weight is not None else [])


def _exact_window(s):
    c = s["case"]
    B, Hq, N, d, G = c["B"], c["Hq"], c["N"], c["d"], c["Hq"] // c["Hkv"]
    o = torch.zeros((B, Hq, N, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Hq, N), dtype=torch.float64, device="cuda")
    nhd = c["layout"] == "NHD"
    lens = [N] * B if s["lens"] is None else s["lens"].tolist()
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        p = torch.arange(n, device="cuda")
        hidden = (p[None] > p[:, None]) | ((p[:, None] - p[None] >= c["window"]) & (p[None] >= c["sinks"]))
        for h in range(Hq):
            q, k, v = ((x[b, :n, y] if nhd else x[b, y, :n]).double()
                       for x, y in ((s["q"], h), (s["k"], h // G), (s["v"], h // G)))
            t = (q @ k.T) / math.sqrt(d)
            t[hidden] = float("-inf")
            z = torch.logsumexp(t, -1, keepdim=True)
            o[b, h, :n] = torch.exp(t - z) @ v
            lse[b, h, :n] = z[:, 0]
    return [o.transpose(1, 2).contiguous() if nhd else o, lse]


def _exact_evict(s):
    c = s["case"]
    page, keep, H = c["page"], c["keep"], c["Hkv"]
    quant = c["cache"] == "8"
    weight = s["weight"].double()
    pools = [None if quant else s["k_pages"].double(), s["v_pages"].double()]
    scales = [s["k_scale"].double(), s["v_scale"].double()] if quant else []
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b].long()
        to = torch.arange(min(n, keep), device="cuda")
        dst, row = s["dst_table"][b].long()[to // page], to % page
        for h in range(H):
            src = torch.arange(n, device="cuda")
            if n > keep:
                w = s["weight"][ids, h].flatten()[c["sinks"]:n - c["recent"]]
                top = torch.sort(-w, stable=True)[1][:keep - c["sinks"] - c["recent"]] + c["sinks"]
                src = torch.cat([src[:c["sinks"]], torch.sort(top)[0], src[n - c["recent"]:]])
            fid, frow = ids[src // page], src % page
            for x in pools:
                if x is not None and c["layout"] == "HND":
                    x[dst, h, row] = x[fid, h, frow]
                elif x is not None:
                    x[dst, row, h] = x[fid, frow, h]
            for x in scales + [weight]:
                x[dst, h, row] = x[fid, h, frow]
    return [None, None, weight] + pools + scales


# ---------------------------------------------------------------- the work
def work(case):
    """Bytes and operations that one call cannot do without."""
    c = case
    d, B = c["d"], c["B"]
    if c["op"] == "window":
        lens = _lengths(B, c["N"] // 2, c["N"]) if c["padded"] else [c["N"]] * B
        pairs = sum(_pairs(n, c["window"], c["sinks"]) for n in lens)
        return {"bytes": float(sum(lens)) * ((2 * c["Hq"] + 2 * c["Hkv"]) * d * 2 + 4 * c["Hq"]),
                "flops": 4.0 * d * c["Hq"] * pairs}
    H = c["Hkv"]
    token = 2 * H * (2 * d if c["cache"] == "16" else d + 4)  # bytes of one cached token, K and V
    if c["op"] == "append":
        n = sum(_new_tokens(c))
        return {"bytes": float(n) * (4 * H * d + token), "flops": 0.0 if c["cache"] == "16" else 6.0 * n * H * d}
    lens = _lengths(B, c["shortest"], c["longest"])
    if c["op"] == "decode":
        seen = sum(_visible(n, c["window"], c["sinks"]) for n in lens)
        return {"bytes": float(seen) * (token + (8 * H if c["track"] else 0)) + B * c["Hq"] * (4 * d + 4),
                "flops": 4.0 * d * c["Hq"] * seen}
    read = sum(n for n in lens if n > c["keep"])
    moved = sum(min(n, c["keep"]) for n in lens)
    return {"bytes": 4.0 * H * read + moved * (2.0 * (token + 4 * H) + 4 * H), "flops": float(H * read)}


def _pairs(n, window, sinks):
    """Visible (query, key) pairs of n rows."""
    w, t = min(n, window), min(sinks, max(0, n - window))
    # rows below the window see all before them; later ones the window and the sinks outside of it
    return w * (w + 1) // 2 + (n - w) * w + t * (t - 1) // 2 + t * max(0, n - window - t + 1) if t else \
        w * (w + 1) // 2 + (n - w) * w
