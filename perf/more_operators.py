"""What the 8-bit KV cache and the paging calls are measured on.

The operators (formulas in the functions below):

- plan_step / release_pages: from the tokens that each request holds and gets,
  its rows in the batch, their lengths and slots, and the pages that it needs,
  taken from the end of a list of free pages; and pages given back to that list.
- append_kv_fp8 / gather_kv_fp8: K and V rows as e4m3 codes with one
  power-of-two scale per block of B tokens and KV head, written into the paged
  cache and read back as BF16.  A block's scale is the smallest 2^e with
  max|x| <= 448 2^e; a block that already holds earlier tokens keeps at least
  its scale, and where that grows, their codes are rounded once more.
- sparse_attn_fp8: softmax attention over the slots a selection returned,
  reading the 8-bit cache.
- window_attn_fp8: a row that sees L tokens attends to the last `window` of
  them and to the first `n_sink` (a window of the context: causal attention).

`own` False: plain torch in FP32, rounded once at the end.  `own` True: the
library's calls.
"""
import math

import numpy as np
import torch

own = False

_qsa = None


def _lib():
    global _qsa
    if _qsa is None:
        import sparse_attention_indexer_index_gb300 as qsa
        _qsa = qsa
    return _qsa


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 requests: its rows, slots and pages, then the step taken back
        dict(name="plan_step_32req", kind="plan", n_req=32, tok_lo=1, tok_hi=1, ctx_lo=4096, ctx_hi=131072, page=64,
             pad=0, shape=1),
        # 1,500 requests of 0 to 6 tokens (decode and verify rows) in a batch padded for a captured graph, small pages
        dict(name="plan_verify_1500req", kind="plan", n_req=1500, tok_lo=0, tok_hi=6, ctx_lo=1, ctx_hi=8191, page=16,
             pad=500, shape=2),
        # 37 prompts and chunks, some 65,000 tokens
        dict(name="plan_prompts_37req", kind="plan", n_req=37, tok_lo=501, tok_hi=3001, ctx_lo=0, ctx_hi=30001, page=64,
             pad=129, shape=3),
        # one decode step of 32 requests writes its tokens' K and V; the blocks it wrote into are read back
        dict(name="kv8_step_32req", kind="kv", n_req=32, tok_lo=1, tok_hi=1, ctx_lo=4096, ctx_hi=131072, h_kv=2, d=256,
             page=64, block=64, shape=4),
        # five prompts of odd lengths written into the cache and read back
        dict(name="kv8_prompts_5req", kind="kv", n_req=5, tok_lo=9001, tok_hi=17003, ctx_lo=0, ctx_hi=4999, h_kv=2,
             d=256, page=64, block=64, shape=5),
        # one request's decode token over its selection
        dict(name="sparse8_1x2051", kind="sparse", n_req=1, rows=1, n_idx=2051, ctx_lo=8192, ctx_hi=8192, h_q=16, h_kv=2,
             d=256, page=64, block=64, shape=6),
        # batched decode: 32 requests of 4K to 131K tokens
        dict(name="sparse8_32x2051", kind="sparse", n_req=32, rows=1, n_idx=2051, ctx_lo=4096, ctx_hi=131072, h_q=16,
             h_kv=2, d=256, page=64, block=64, shape=7),
        # 32 verify steps of 6 rows at 80,000 tokens, one KV head for all query heads
        dict(name="sparse8_192x2051_d128", kind="sparse", n_req=32, rows=6, n_idx=2051, ctx_lo=80000, ctx_hi=80000,
             h_q=16, h_kv=1, d=128, page=64, block=32, shape=8),
        # one decode token of a full-attention layer
        dict(name="causal8_step_1req", kind="window", n_req=1, row_lo=1, row_hi=1, ctx_lo=20011, ctx_hi=20011,
             window=131072, n_sink=0, h_q=16, h_kv=2, d=256, page=64, block=64, shape=9),
        # batched decode in a window layer
        dict(name="window8_step_32req", kind="window", n_req=32, row_lo=1, row_hi=1, ctx_lo=4096, ctx_hi=131072,
             window=4096, n_sink=4, h_q=16, h_kv=2, d=256, page=64, block=64, shape=10),
        # verify steps of 32 requests (6 rows each) in a window layer
        dict(name="window8_verify_32x6", kind="window", n_req=32, row_lo=6, row_hi=6, ctx_lo=4096, ctx_hi=131072,
             window=1024, n_sink=4, h_q=16, h_kv=2, d=256, page=64, block=64, shape=11),
        # batched decode of a full-attention layer: 8 requests of up to 131,072 tokens, small pages
        dict(name="causal8_step_8req", kind="window", n_req=8, row_lo=1, row_hi=2, ctx_lo=65537, ctx_hi=131072,
             window=131072, n_sink=0, h_q=16, h_kv=4, d=128, page=16, block=16, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "kv", "sparse", "window", "window"])
    h_q, h_kv, d = rng.choice([(16, 2, 256), (8, 2, 256), (16, 1, 128), (16, 4, 128), (8, 4, 128), (16, 2, 128)])
    page = rng.choice([16, 32, 64, 64, 128])
    c = dict(kind=kind, page=page, shape=rng.randrange(1 << 20))
    if kind == "plan":
        n = _log(rng, 1, 2000)
        hi = _log(rng, 1, max(1, 65000 // n))
        c.update(n_req=n, tok_lo=rng.choice([0, hi // 2]), tok_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 16, 20000),
                 pad=rng.choice([0, 7, 300]))
        return c
    c.update(h_kv=h_kv, d=d, block=rng.choice([b for b in (16, 32, 64, 128) if page % b == 0]))
    if kind == "kv":
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 65000 // n))
        c.update(n_req=n, tok_lo=max(1, hi // 2), tok_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 16, 20000))
    elif kind == "sparse":
        n = _log(rng, 1, 48)
        c.update(n_req=n, rows=rng.choice([1, 1, 2, 4]), n_idx=_log(rng, 32, 2051), ctx_lo=_log(rng, 1, 4096),
                 ctx_hi=_log(rng, 4097, 80000), h_q=h_q)
    elif rng.random() < 0.6:  # window layers: decode and verify rows
        c.update(window=_log(rng, 64, 4096), n_sink=rng.choice([0, 1, 4, 16, 65]), h_q=h_q, n_req=_log(rng, 1, 48),
                 row_lo=1, row_hi=rng.choice([1, 1, 4, 6, 8]), ctx_lo=_log(rng, 1, 4096), ctx_hi=_log(rng, 4097, 80000))
    else:  # full-attention layers, up to about the largest listed work
        n = _log(rng, 1, 16)
        hi = _log(rng, 300, 350000000 // (n * h_kv * d))
        c.update(window=131072, n_sink=rng.choice([0, 4]), h_q=h_q, n_req=n, row_lo=1, row_hi=rng.choice([1, 1, 2, 6]),
                 ctx_lo=min(hi, 131072) // 3, ctx_hi=min(hi, 131072))
    return c


def _shapes(c):
    """Tokens or rows per request, tokens before them (None for rows) and after
    them, from the case's `shape` number alone."""
    r = np.random.default_rng(c["shape"])
    if c["kind"] in ("plan", "kv"):
        n = r.integers(c["tok_lo"], c["tok_hi"] + 1, c["n_req"])
        first = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, c["n_req"])
        return n, first, first + n
    ctx = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, c["n_req"])
    n = np.full(c["n_req"], c["rows"]) if c["kind"] == "sparse" else r.integers(c["row_lo"], c["row_hi"] + 1, c["n_req"])
    return n, None, np.maximum(ctx, n)


def _rows(n, ctx):
    """Row lengths: request r's rows are its last n[r] tokens."""
    return np.concatenate([np.arange(e - m + 1, e + 1) for m, e in zip(n, ctx)])


def _pairs(c):
    """(row, key) pairs of a window case, and distinct keys read per request."""
    n, _, ctx = _shapes(c)
    L = _rows(n, ctx)
    lo = np.maximum(L - c["window"], 0)
    seen = L - lo + np.minimum(lo, c["n_sink"])
    klo = np.maximum(ctx - n + 1 - c["window"], 0)
    keys = ctx - klo + np.minimum(klo, c["n_sink"])
    return int(seen.sum()), int(keys.sum()), int(n.sum())


def _old(c):
    """Earlier tokens in the blocks that a step writes into, in all."""
    return int((_shapes(c)[1] % c["block"]).sum())


def work(c):
    if c["kind"] == "plan":
        n, first, _ = _shapes(c)
        new = int(((first + n + c["page"] - 1) // c["page"] - (first + c["page"] - 1) // c["page"]).sum())
        t = int(n.sum()) + c["pad"]
        # lengths read; starts and lengths written; four words a row; a page moves to the table and back
        return {"bytes": 4 * (2 * c["n_req"] + 2 * c["n_req"] + 1 + 3 * t + 4 * new), "flops": 6 * t}
    row8 = 2 * c["h_kv"] * c["d"]  # K and V of a token in 8 bits
    row16 = 2 * row8
    if c["kind"] == "kv":
        t, b = int(_shapes(c)[0].sum()), _old(c)
        # append: BF16 read, codes written; read back: the reverse, with the blocks' earlier tokens
        return {"bytes": t * (row16 + row8) + (t + b) * (row16 + row8), "flops": (2 * t + b) * row8 * 2}
    if c["kind"] == "sparse":
        rows = c["n_req"] * c["rows"]
        pairs = int(np.minimum(_rows(*_shapes(c)[::2]), c["n_idx"]).sum())
        # rows of one request select nearly the same slots, but each its own list
        return {"bytes": pairs * row8 + rows * (c["n_idx"] * 4 + c["h_q"] * (c["d"] * 6 + 4)),
                "flops": 4 * pairs * c["h_q"] * c["d"]}
    pairs, keys, rows = _pairs(c)
    return {"bytes": keys * row8 + rows * c["h_q"] * (c["d"] * 4 + 4), "flops": 4 * pairs * c["h_q"] * c["d"]}


# ------------------------------------------------------------- 8-bit blocks
def _exponent(top):
    """Smallest e with top <= 448 2^e, between -64 and 63 (exact: top = m 2^k, 448 = 0.875 2^9)."""
    m, k = torch.frexp(top)
    e = k - 9 + (m > 0.875).to(k.dtype)
    return torch.where(top > 0, e.clamp(-64, 63), torch.full_like(e, -64))


def _pow2(e):
    """2^e in FP32, from its bits (e between -126 and 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, e):
    """e4m3 codes of x / 2^e (nearest even, saturating), uint8."""
    y = (x.float() * _pow2(-e)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, scales):
    """FP32 values of codes [..., d] under scale bytes [...] (2^(byte - 127))."""
    return codes.view(torch.float8_e4m3fn).float() * _pow2(scales.to(torch.int32) - 127)[..., None]


# ------------------------------------------------------------------- inputs
def _pages(gen, ctx, page, dev):
    """A page table covering ctx, its pages a random permutation of the pool."""
    n = [(int(e) + page - 1) // page for e in ctx]
    total, width = sum(n) + 3, max(1, max(n))
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    off = np.concatenate([[0], np.cumsum(n)])
    pt = torch.zeros((len(n), width), dtype=torch.int32, device=dev)
    for r, m in enumerate(n):
        pt[r, :m] = perm[off[r]:off[r] + m]
    return pt, total * page


def _bank(gen, n, h_kv, d, dev, kind):
    """K or V rows: normal, a few strong channels in K, V smaller; magnitudes vary from token to token."""
    x = torch.randn((n, h_kv, d), generator=gen, device=dev)
    if kind == "k":
        gain = torch.ones(d, device=dev)
        gain[torch.randperm(d, generator=gen, device=dev)[:d // 32]] = 5.0
        x = x * gain
    else:
        x = x * 0.4 * torch.exp(0.5 * torch.randn((n, 1, 1), generator=gen, device=dev))
    return x.to(torch.bfloat16)


def _cache(gen, n_slots, block, h_kv, d, dev, kind):
    """A cache of n_slots rows: codes and scale bytes, blocks drawn from 16,384 rows' worth."""
    x = _bank(gen, 16384, h_kv, d, dev, kind).unflatten(0, (-1, block))
    e = _exponent(x.float().abs().amax((1, 3)))
    codes = _codes(x, e[:, None, :, None])
    pick = torch.randint(0, x.shape[0], (n_slots // block,), generator=gen, device=dev)
    return codes[pick].flatten(0, 1), (e + 127).to(torch.uint8)[pick]


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + c["shape"])
    page = c["page"]
    n, first, ctx = _shapes(c)
    start = np.concatenate([[0], np.cumsum(n)])
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    if c["kind"] == "plan":
        # the pages of the tokens that are there, and a list of free ones that covers the step with a few over
        held = (first + page - 1) // page
        need = int(((ctx + page - 1) // page - held).sum())
        pool = int(held.sum()) + need + 17
        perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        width = int(((ctx + page - 1) // page).max()) + 1
        pt = torch.full((len(n), width), -1, dtype=torch.int32, device=dev)
        col = torch.arange(width, device=dev)[None]
        pt[col < i32(held)[:, None]] = perm[:int(held.sum())]
        free = torch.full((pool,), -1, dtype=torch.int32, device=dev)
        free[:need + 17] = perm[int(held.sum()):]
        t = int(start[-1]) + c["pad"]
        return dict(kind="plan", page=page, pt=pt, free=free, n_free=i32([need + 17]), ctx=i32(first), n_new=i32(n), n_tok=t,
                    from_page=i32(held), to_page=i32((ctx + page - 1) // page),
                    start=torch.empty(len(n) + 1, dtype=torch.int32, device=dev),
                    new_len=torch.empty(len(n), dtype=torch.int32, device=dev),
                    row_len=torch.empty(t, dtype=torch.int32, device=dev),
                    row_req=torch.empty(t, dtype=torch.int32, device=dev),
                    slots=torch.empty(t, dtype=torch.int32, device=dev))
    h_kv, d, block = c["h_kv"], c["d"], c["block"]
    pt, n_slots = _pages(gen, ctx, page, dev)
    s = dict(kind=c["kind"], pt=pt, page=page, block=block, n_slots=n_slots, h_kv=h_kv, d=d)
    s["kc"], s["ks"] = _cache(gen, n_slots, block, h_kv, d, dev, "k")
    s["vc"], s["vs"] = _cache(gen, n_slots, block, h_kv, d, dev, "v")
    if c["kind"] == "kv":
        t = int(start[-1])
        k_new, v_new = _bank(gen, t, h_kv, d, dev, "k"), _bank(gen, t, h_kv, d, dev, "v")
        # the slots of every touched block up to the request's last token
        begin = first // block * block
        pos = torch.as_tensor(np.concatenate([np.arange(b, e) for b, e in zip(begin, ctx)]), device=dev)
        req = torch.as_tensor(np.repeat(np.arange(len(n)), ctx - begin), device=dev)
        slots = (pt[req, pos // page].long() * page + pos % page).to(torch.int32)
        s.update(k_new=k_new, v_new=v_new, start=i32(start), first=i32(first), slots=slots,
                 k_out=torch.empty((len(pos), h_kv, d), dtype=torch.bfloat16, device=dev),
                 v_out=torch.empty((len(pos), h_kv, d), dtype=torch.bfloat16, device=dev))
        return s
    L = _rows(n, ctx)
    rows, h_q = len(L), c["h_q"]
    req = torch.as_tensor(np.repeat(np.arange(len(n)), n), device=dev)
    if c["kind"] == "sparse":
        # a selection: runs of 4 consecutive positions, ascending, as many as the row has
        w, run = c["n_idx"], 4
        nb = -(-w // run)
        Lt = torch.as_tensor(L, device=dev)
        blocks = (Lt // run).clamp(min=1)
        at = torch.linspace(0, 1, nb + 1, device=dev, dtype=torch.float64)[:nb]
        jit = torch.rand((rows, nb), generator=gen, device=dev, dtype=torch.float64) / (nb + 1)
        b = ((at[None] + jit) * blocks[:, None]).long().clamp(max=blocks[:, None] - 1)
        few = blocks[:, None] <= nb
        b = torch.where(few, torch.arange(nb, device=dev)[None].expand(rows, nb), b)
        p = (b[:, :, None] * run + torch.arange(run, device=dev)).flatten(1)[:, :w]
        slots = pt[req[:, None], (p.clamp(max=int(max(ctx)) - 1) // page)].long() * page + p % page
        s["slots"] = torch.where(p >= Lt[:, None], torch.full_like(slots, -1), slots).to(torch.int32).contiguous()
    else:
        s.update(window=c["window"], n_sink=c["n_sink"], start=i32(start), row_len=i32(L), req=req,
                 max_len=int(max(ctx)), max_rows=int(max(n)), ctx=torch.as_tensor(ctx, device=dev))
    s["q"] = torch.randn((rows, h_q, d), generator=gen, device=dev).to(torch.bfloat16)
    s["scale"] = d ** -0.5
    s["out"] = torch.empty((rows, h_q, d), dtype=torch.float32 if c["kind"] == "sparse" else torch.bfloat16, device=dev)
    s["lse"] = torch.empty((rows, h_q), dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------- runs
def _plain_plan(s):
    dev, page, pt, free = s["pt"].device, s["page"], s["pt"], s["free"]
    ctx, n = s["ctx"].long(), s["n_new"].long()
    i = torch.arange(s["n_tok"], device=dev)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(n, 0)])
    held, end = (ctx + page - 1) // page, (ctx + n + page - 1) // page
    last = torch.cumsum(end - held, 0)            # pages taken by the requests up to this one
    base = s["n_free"].long() - last[-1]          # they are the end of the list, in the requests' order
    col = torch.arange(pt.shape[1], device=dev)[None]
    fresh = (col >= held[:, None]) & (col < end[:, None])
    at = base + (last - (end - held))[:, None] + col - held[:, None]
    pt.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], pt))
    r = torch.searchsorted(start[1:].contiguous(), i, right=True)
    real = i < start[-1]
    rr = r.clamp(max=n.numel() - 1)
    pos = ctx[rr] + i - start[rr]
    slot = pt[rr, (pos // page).clamp(0, pt.shape[1] - 1)].long() * page + pos % page
    s["start"].copy_(start)
    s["new_len"].copy_(ctx + n)
    s["row_len"].copy_(torch.where(real, pos + 1, torch.zeros_like(pos)))
    s["row_req"].copy_(torch.where(real, rr, torch.full_like(rr, -1)))
    s["slots"].copy_(torch.where(real, slot, torch.full_like(slot, -1)))
    s["n_free"].copy_(base)
    # the step taken back: its pages go to the end of the list again
    begin, stop = s["from_page"].long()[:, None], s["to_page"].long()[:, None]
    back = (col >= begin) & (col < stop) & (pt >= 0)
    rank = torch.cumsum(back.flatten().long(), 0) - 1
    total = rank[-1:] + 1
    j = torch.arange(free.numel(), device=dev) - s["n_free"].long()
    order = torch.searchsorted(rank + 1, j + 1).clamp(max=rank.numel() - 1)  # the j-th entry given back
    free.copy_(torch.where((j >= 0) & (j < total), pt.flatten()[order], free))
    pt.copy_(torch.where(back, torch.full_like(pt, -1), pt))
    s["n_free"].copy_(s["n_free"].long() + total)
    return tuple(s[k] for k in ("start", "new_len", "row_len", "row_req", "slots", "pt", "free", "n_free"))


def _plain_append(s, new, codes, scales, pos, slot, old, old_block):
    """New rows [t][h][d] into codes / scales: pos and slot of every new token,
    slots of the earlier tokens in the touched blocks and what was there."""
    block, h = s["block"], s["h_kv"]
    top = new.float().abs().amax(-1)                                       # [t][h]
    b = slot // block
    most = torch.zeros((scales.shape[0], h), device=top.device).scatter_reduce_(0, b[:, None].expand(-1, h), top, "amax")
    opened = torch.zeros(scales.shape[0], dtype=torch.bool, device=top.device)
    opened[b[pos % block == 0]] = True                                     # the block's first token is in this step
    touched = torch.zeros_like(opened)
    touched[b] = True
    before = scales.to(torch.int32) - 127
    e = _exponent(most)
    e = torch.where(opened[:, None], e, torch.maximum(e, before))
    e = torch.where(touched[:, None], e, before)
    codes[old] = _codes(_values(codes[old], scales[old_block]), e[old_block][..., None])
    codes[slot] = _codes(new, e[b][..., None])
    scales.copy_((e + 127).to(torch.uint8))


def _plain_kv(s):
    page, block, pt = s["page"], s["block"], s["pt"]
    dev, t = pt.device, s["k_new"].shape[0]
    i = torch.arange(t, device=dev)
    r = torch.searchsorted(s["start"][1:].contiguous(), i.to(torch.int32), right=True)
    pos = s["first"][r].long() + i - s["start"][r]
    slot = pt[r, pos // page].long() * page + pos % page
    # earlier tokens of the requests' first blocks
    o = torch.arange(block, device=dev)[None]
    first = s["first"].long()[:, None]
    p = first // block * block + o
    n = (s["start"][1:] - s["start"][:-1])[:, None]
    rows, cols = torch.nonzero((p < first) & (n > 0), as_tuple=True)
    p = p[rows, cols]
    old = pt[rows, p // page].long() * page + p % page
    _plain_append(s, s["k_new"], s["kc"], s["ks"], pos, slot, old, old // block)
    _plain_append(s, s["v_new"], s["vc"], s["vs"], pos, slot, old, old // block)
    at = s["slots"].long()
    return (_values(s["kc"][at], s["ks"][at // block]).to(torch.bfloat16),
            _values(s["vc"][at], s["vs"][at // block]).to(torch.bfloat16))


def _softmax_rows(logit, v, eq):
    """Attention weights of masked (-inf) logits times v; empty rows give 0 and -inf."""
    m = logit.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(logit - m)
    z = e.sum(-1, keepdim=True)
    o = torch.einsum(eq, torch.where(z > 0, e / z, torch.zeros_like(e)), v)
    return o, (m + torch.log(z))[..., 0]


def _plain_slots(s, codes, scales, slots):
    at = slots.long().clamp(min=0)
    return torch.where((slots >= 0)[..., None, None], _values(codes[at], scales[at // s["block"]]),
                       torch.zeros((), device=slots.device))


def _plain(s):
    k = s["kind"]
    if k == "plan":
        return _plain_plan(s)
    if k == "kv":
        return _plain_kv(s)
    h_kv = s["h_kv"]
    if k == "sparse":
        kk, vv = _plain_slots(s, s["kc"], s["ks"], s["slots"]), _plain_slots(s, s["vc"], s["vs"], s["slots"])
        q = s["q"].float().unflatten(1, (h_kv, -1))
        logit = torch.einsum("thgd,tjhd->thgj", q, kk) * s["scale"]
        logit = torch.where((s["slots"] >= 0)[:, None, None], logit, torch.full_like(logit, -math.inf))
        o, lse = _softmax_rows(logit, vv, "thgj,tjhd->thgd")
        return o.flatten(1, 2), lse.flatten(1, 2)
    # window: each request's keys from its first row's window to its end, and the sinks
    dev, W, S, page = s["pt"].device, s["window"], s["n_sink"], s["page"]
    ctx, n_req = s["ctx"], s["ctx"].numel()
    span = min(s["max_len"], W + s["max_rows"] - 1)
    p = (ctx - span)[:, None] + torch.arange(span, device=dev)[None]
    p = torch.cat([torch.arange(S, device=dev)[None].expand(n_req, S), p], 1)
    real = p >= 0
    real[:, :S] = p[:, :S] < (ctx - span).clamp(min=0)[:, None]
    pc = p.clamp(min=0)
    page_of = torch.gather(s["pt"].long(), 1, (pc // page).clamp(max=s["pt"].shape[1] - 1))
    slots = torch.where(real, page_of * page + pc % page, torch.full_like(pc, -1))
    kk, vv = _plain_slots(s, s["kc"], s["ks"], slots), _plain_slots(s, s["vc"], s["vs"], slots)
    # rows padded to [request][row]
    i = torch.arange(s["max_rows"], device=dev)[None]
    count = (s["start"][1:] - s["start"][:-1])[:, None]
    at = (s["start"][:-1, None] + i).clamp(max=s["row_len"].numel() - 1).long()
    L = torch.where(i < count, s["row_len"][at], torch.zeros((), dtype=torch.int32, device=dev))
    q = s["q"].float()[at].unflatten(2, (h_kv, -1))
    logit = torch.einsum("rthgd,rjhd->rhgtj", q, kk) * s["scale"]
    seen = real[:, None] & (p[:, None] < L[..., None]) & ((p[:, None] >= L[..., None] - W) | (p[:, None] < S))
    logit = torch.where(seen[:, None, None], logit, torch.full((), -math.inf, device=dev))
    o, lse = _softmax_rows(logit, vv, "rhgtj,rjhd->rthgd")
    back = torch.arange(s["row_len"].numel(), device=dev) - s["start"].long()[s["req"]]
    return o.flatten(2, 3)[s["req"], back].to(torch.bfloat16), lse.permute(0, 3, 1, 2).flatten(2, 3)[s["req"], back]


def run(s):
    if not own:
        return _plain(s)
    qsa, k = _lib(), s["kind"]
    if k == "plan":
        rows = qsa.plan_step(s["ctx"], s["n_new"], s["pt"], s["page"], s["free"], s["n_free"], s["n_tok"],
                             req_row_start=s["start"], new_len=s["new_len"], row_len=s["row_len"], row_req=s["row_req"],
                             slots=s["slots"])
        return (*rows, *qsa.release_pages(s["pt"], s["from_page"], s["to_page"], s["free"], s["n_free"]))
    if k == "kv":
        qsa.append_kv_fp8(s["k_new"], s["v_new"], s["start"], s["first"], s["kc"], s["ks"], s["vc"], s["vs"], s["pt"],
                          s["page"])
        return qsa.gather_kv_fp8(s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    if k == "sparse":
        return qsa.sparse_attn_fp8(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], s["scale"], out=s["out"],
                                   lse=s["lse"])
    return qsa.window_attn_fp8(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["start"], s["row_len"], s["pt"], s["page"],
                               s["max_len"], s["window"], s["n_sink"], s["scale"], max_rows_per_req=s["max_rows"],
                               out=s["out"], lse=s["lse"])


# --------------------------------------------------------------------- exact
def _two(e):
    """2^e in FP64."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _read64(codes, scales):
    """Values in FP64, decoded from the bits: e4m3 = (-1)^s (m + 8 [e > 0]) 2^(max(e, 1) - 10), scale 2^(byte - 127)."""
    u = codes.to(torch.int64)
    e, m = u // 8 % 16, u % 8
    v = (m + 8 * (e > 0)).double() * _two(e.clamp(min=1) - 10) * (1 - 2 * (u // 128)).double()
    return v * _two(scales.long() - 127)[..., None]


def _round64(x, unit):
    """x / unit rounded to the nearest multiple of its e4m3 step (ties to even), times unit, in FP64."""
    a = (x.abs() / unit).clamp(max=448.0)
    step = _two(torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 4)  # 2^(floor(log2 a) - 3)
    return torch.sign(x) * torch.round(a / step) * step * unit


def _unit64(top):
    """Smallest power of two with top <= 448 of it, from 2^-64 to 2^63."""
    e = torch.frexp(top.clamp(min=1e-300) / 448.0).exponent.long()  # below 2^e, from 2^(e - 1) on
    e = torch.where(top <= 448.0 * _two(e - 1), e - 1, e)
    return _two(e.clamp(-64, 63))


def _exact_plan(c, s):
    """Request by request, as a host program would keep its lists."""
    n, first, ctx = _shapes(c)
    page, t = c["page"], s["n_tok"]
    pt, free = s["pt"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    n_free = int(s["n_free"])
    need = [-(-int(e) // page) - -(-int(f) // page) for f, e in zip(first, ctx)]
    take = n_free - sum(need)
    row_len, row_req, slots = np.zeros(t, np.int32), np.full(t, -1, np.int32), np.full(t, -1, np.int32)
    i = 0
    for r in range(len(n)):
        pages = list(pt[r, :-(-int(first[r]) // page)]) + list(free[take:take + need[r]])
        take += need[r]
        for p in range(int(first[r]), int(ctx[r])):
            row_len[i], row_req[i], slots[i] = p + 1, r, pages[p // page] * page + p % page
            i += 1
    start = np.concatenate([[0], np.cumsum(n)])
    return tuple(torch.as_tensor(np.asarray(x, np.int32)) for x in
                 (start, ctx, row_len, row_req, slots, pt, free, [n_free]))


def _exact_kv(c, s):
    n, first, ctx = _shapes(c)
    page, block = c["page"], c["block"]
    outs = []
    for new, codes, scales in ((s["k_new"], s["kc"], s["ks"]), (s["v_new"], s["vc"], s["vs"])):
        got, t = [], 0
        for r, (m, f) in enumerate(zip(n, first)):
            m, f = int(m), int(f)
            rows = new[t:t + m].double()
            t += m
            lo, done = f // block * block, 0
            if lo < f:  # the block that holds earlier tokens
                at = int(s["pt"][r, lo // page]) * page + lo % page
                k = min(m, lo + block - f)
                was = _two(scales[at // block].long() - 127)[:, None]
                unit = torch.maximum(was, _unit64(rows[:k].abs().amax((0, 2)))[:, None])
                kept = _read64(codes[at:at + f - lo], scales[at // block][None])
                got += [_round64(kept, unit), _round64(rows[:k], unit)]
                done = k
            whole = (m - done) // block * block
            if whole:
                x = rows[done:done + whole].unflatten(0, (-1, block))
                got.append(_round64(x, _unit64(x.abs().amax((1, 3)))[:, None, :, None]).flatten(0, 1))
            if done + whole < m:
                x = rows[done + whole:]
                got.append(_round64(x, _unit64(x.abs().amax((0, 2)))[:, None]))
        outs.append(torch.cat(got))
    return tuple(outs)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "plan":
        return _exact_plan(c, s)
    if c["kind"] == "kv":
        return _exact_kv(c, s)
    n, _, ctx = _shapes(c)
    L, h_q, h_kv, d, block = _rows(n, ctx), c["h_q"], c["h_kv"], c["d"], c["block"]
    grp, dev = h_q // h_kv, s["pt"].device
    out = torch.zeros((len(L), h_q, d), dtype=torch.float64, device=dev)
    lse = torch.full((len(L), h_q), -math.inf, dtype=torch.float64, device=dev)

    def attend(t0, t1, slots, seen):
        kk, vv = _read64(s["kc"][slots], s["ks"][slots // block]), _read64(s["vc"][slots], s["vs"][slots // block])
        for h in range(h_q):
            x = s["q"][t0:t1, h].double() @ kk[:, h // grp].T * float(np.float32(s["scale"]))
            x = x.masked_fill(~seen, -math.inf)
            lse[t0:t1, h] = torch.logsumexp(x, -1)
            w = torch.exp(x - lse[t0:t1, h, None]).nan_to_num(0.0)
            out[t0:t1, h] = w @ vv[:, h // grp]

    if c["kind"] == "sparse":
        for t in range(len(L)):
            at = s["slots"][t].long()
            at = at[at >= 0]
            attend(t, t + 1, at, torch.ones((1, at.numel()), dtype=torch.bool, device=dev))
        return out, lse
    t0 = 0
    for r, (m, e) in enumerate(zip(n, ctx)):
        pos = np.arange(e)
        pos = torch.as_tensor(pos[(pos < c["n_sink"]) | (pos >= e - m + 1 - c["window"])], device=dev)
        slots = s["pt"][r].long()[pos // c["page"]] * c["page"] + pos % c["page"]
        Lr = torch.as_tensor(L[t0:t0 + m], device=dev)[:, None]
        attend(t0, t0 + m, slots, (pos < Lr) & ((pos >= Lr - c["window"]) | (pos < c["n_sink"])))
        t0 += m
    return out, lse
