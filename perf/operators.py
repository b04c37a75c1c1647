"""What the 4-bit KV cache and the window attention are measured on.

The operators (formulas in the functions below):

- append_kv_fp4 / gather_kv_fp4: K and V rows quantised to 4 bits as they are
  written into the paged cache, and read back as BF16.  Blocks of 16 values:
  scale = e4m3(max|x| / (6 g)), code = e2m1(x / (scale g)), value = code scale g,
  with g the caller's scale of the whole tensor, a power of two (so that
  every step but the two roundings is exact, and the value fits BF16).
- sparse_attn_fp4: softmax attention over the slots a selection returned,
  reading the 4-bit cache.
- window_attn / window_attn_fp4: a row that sees L tokens attends to the last
  `window` of them and to the first `n_sink`, through the page table, over the
  BF16 or the 4-bit cache.

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
        # one decode step of 32 requests writes its tokens' K and V, then reads them back
        dict(name="kv_step_32req", kind="kv", n_req=32, tok_lo=1, tok_hi=1, ctx_lo=4096, ctx_hi=131072, h_kv=2, d=256,
             page=64, shape=1),
        # five prompts of odd lengths written into the cache and read back
        dict(name="kv_prompts_5req", kind="kv", n_req=5, tok_lo=9001, tok_hi=17003, ctx_lo=0, ctx_hi=4999, h_kv=2, d=256,
             page=64, shape=2),
        # the rows that a 6-row verify step selected, read back (-1 padding among them)
        dict(name="gather_selected_6x2051", kind="gather", n_rows=6, n_idx=2051, ctx=80000, run=4, holes=0.02, h_kv=2,
             d=256, page=64, shape=3),
        # a whole context read back, e.g. to run a prompt's attention in BF16
        dict(name="gather_context_131072", kind="gather", n_rows=1, n_idx=131072, ctx=131072, run=64, holes=0.0, h_kv=4,
             d=128, page=64, shape=4),
        # one request's decode token over its selection
        dict(name="sparse_1x2051", kind="sparse", n_req=1, rows=1, n_idx=2051, ctx_lo=8192, ctx_hi=8192, h_q=16, h_kv=2,
             d=256, page=64, shape=5),
        # batched decode: 32 requests of 4K to 131K tokens
        dict(name="sparse_32x2051", kind="sparse", n_req=32, rows=1, n_idx=2051, ctx_lo=4096, ctx_hi=131072, h_q=16,
             h_kv=2, d=256, page=64, shape=6),
        # 32 verify steps of 6 rows at 80,000 tokens, one KV head for all query heads
        dict(name="sparse_192x2051_d128", kind="sparse", n_req=32, rows=6, n_idx=2051, ctx_lo=80000, ctx_hi=80000, h_q=16,
             h_kv=1, d=128, page=64, shape=7),
        # one decode token in a window layer
        dict(name="window_step_1req", kind="window", fp4=False, n_req=1, row_lo=1, row_hi=1, ctx_lo=8192, ctx_hi=8192,
             window=1024, n_sink=4, h_q=16, h_kv=2, d=256, page=64, shape=8),
        # batched decode in a window layer over the 4-bit cache
        dict(name="window_step_32req_fp4", kind="window", fp4=True, n_req=32, row_lo=1, row_hi=1, ctx_lo=4096,
             ctx_hi=131072, window=4096, n_sink=4, h_q=16, h_kv=2, d=256, page=64, shape=9),
        # verify steps of 32 requests (6 rows each) in a window layer
        dict(name="window_verify_32x6", kind="window", fp4=False, n_req=32, row_lo=6, row_hi=6, ctx_lo=4096,
             ctx_hi=131072, window=1024, n_sink=4, h_q=16, h_kv=2, d=256, page=64, shape=10),
        # a prefill chunk at the end of a 131,072-token context
        dict(name="window_chunk_4096", kind="window", fp4=False, n_req=1, row_lo=4096, row_hi=4096, ctx_lo=131072,
             ctx_hi=131072, window=1024, n_sink=4, h_q=16, h_kv=2, d=256, page=64, shape=11),
        # seven prompts of 1 to 2,000 tokens in one batch, small pages
        dict(name="window_prompts_7req_d128", kind="window", fp4=False, n_req=7, row_lo=1, row_hi=2003, ctx_lo=0,
             ctx_hi=0, window=500, n_sink=1, h_q=16, h_kv=4, d=128, page=16, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["kv", "gather", "sparse", "window", "window"])
    h_q, h_kv, d = rng.choice([(16, 2, 256), (8, 2, 256), (16, 1, 128), (16, 4, 128), (8, 4, 128), (16, 2, 128)])
    c = dict(kind=kind, h_kv=h_kv, d=d, page=rng.choice([16, 32, 64, 64, 128]), shape=rng.randrange(1 << 20))
    if kind == "kv":
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 65000 // n))
        c.update(n_req=n, tok_lo=max(1, hi // 2), tok_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 16, 20000))
    elif kind == "gather":
        rows = _log(rng, 1, 64)
        n_idx = _log(rng, 16, 131072 // rows)
        c.update(n_rows=rows, n_idx=n_idx, ctx=n_idx + _log(rng, 64, 80000), run=rng.choice([1, 4, 64]),
                 holes=rng.choice([0.0, 0.05]))
    elif kind == "sparse":
        n = _log(rng, 1, 48)
        c.update(n_req=n, rows=rng.choice([1, 1, 2, 4]), n_idx=_log(rng, 32, 2051), ctx_lo=_log(rng, 1, 4096),
                 ctx_hi=_log(rng, 4097, 80000), h_q=h_q)
    else:
        w = _log(rng, 64, 4096)
        c.update(window=w, n_sink=rng.choice([0, 1, 4, 16, 65]), h_q=h_q)
        if rng.random() < 0.5:  # decode and verify rows
            hi = rng.choice([1, 1, 6])
            c.update(fp4=rng.random() < 0.5, n_req=_log(rng, 1, 48), row_lo=1, row_hi=hi, ctx_lo=_log(rng, 1, 4096),
                     ctx_hi=_log(rng, 4097, 80000))
        else:  # prompts and chunks, up to about the largest listed work
            n = _log(rng, 1, 8)
            hi = _log(rng, 9, max(10, min(2048, 4096 * 1024 // (w + 16)) // n))
            c.update(fp4=False, n_req=n, row_lo=max(1, hi // 3), row_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 16, 40000))
    return c


def _shapes(c):
    """The lengths that a case stands for, from its `shape` number alone."""
    r = np.random.default_rng(c["shape"])
    k = c["kind"]
    if k == "kv":
        n = r.integers(c["tok_lo"], c["tok_hi"] + 1, c["n_req"])
        first = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, c["n_req"])
        return n, first, first + n
    if k == "gather":
        return np.array([c["n_idx"]] * c["n_rows"]), None, np.array([c["ctx"]] * c["n_rows"])
    ctx = r.integers(c["ctx_lo"], c["ctx_hi"] + 1, c["n_req"])
    if k == "sparse":
        n = np.full(c["n_req"], c["rows"])
        return n, None, np.maximum(ctx, c["rows"])
    n = r.integers(c["row_lo"], c["row_hi"] + 1, c["n_req"])
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


def work(c):
    row4 = 2 * c["h_kv"] * (c["d"] // 2 + c["d"] // 16)  # K and V of a token in 4 bits
    row16 = 2 * c["h_kv"] * c["d"] * 2
    if c["kind"] == "kv":
        t = int(_shapes(c)[0].sum())
        # append: BF16 read, codes and scales written; read back: the reverse
        return {"bytes": t * 2 * (row16 + row4), "flops": t * 2 * c["h_kv"] * c["d"] * 4}
    if c["kind"] == "gather":
        t = c["n_rows"] * c["n_idx"]
        return {"bytes": t * (row16 + row4 + 4), "flops": t * 2 * c["h_kv"] * c["d"]}
    if c["kind"] == "sparse":
        rows = c["n_req"] * c["rows"]
        per = np.minimum(_rows(*_shapes(c)[::2]), c["n_idx"])
        pairs = int(per.sum())
        # rows of one request select nearly the same slots, but each its own list
        return {"bytes": pairs * row4 + rows * (c["n_idx"] * 4 + c["h_q"] * (c["d"] * 6 + 4)),
                "flops": 4 * pairs * c["h_q"] * c["d"]}
    pairs, keys, rows = _pairs(c)
    return {"bytes": keys * (row4 if c["fp4"] else row16) + rows * c["h_q"] * (c["d"] * 4 + 4),
            "flops": 4 * pairs * c["h_q"] * c["d"]}


# ------------------------------------------------------------- 4-bit blocks
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
K_SCALE, V_SCALE = 2.0 ** -6, 2.0 ** -7  # the tensors' own scales, as a calibration would set them


def _quantise(x, g):
    """x [..., d] -> (codes [..., d/2] uint8, low nibble first; scales [..., d/16] e4m3 bytes)."""
    b = x.float().unflatten(-1, (-1, 16))
    g = torch.tensor(g, dtype=torch.float32, device=x.device)
    s8 = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    eff = s8.float() * g
    a = torch.where(eff[..., None] > 0, b.abs() / eff[..., None], torch.zeros_like(b))
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    n = (m + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2)
    return n[..., 0::2] + 16 * n[..., 1::2], s8.view(torch.uint8)


def _values(codes, scales, g):
    """The FP32 values that codes and scales stand for."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * torch.tensor(g, dtype=torch.float32, device=codes.device)


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


def _bank(gen, h_kv, d, dev, kind):
    """16,384 K or V rows: normal, a few strong channels in K, V smaller."""
    x = torch.randn((16384, h_kv, d), generator=gen, device=dev)
    if kind == "k":
        gain = torch.ones(d, device=dev)
        gain[torch.randperm(d, generator=gen, device=dev)[:d // 32]] = 5.0
        x = x * gain
    else:
        x = x * 0.4
    return x.to(torch.bfloat16)


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + c["shape"])
    h_kv, d, page = c["h_kv"], c["d"], c["page"]
    n, first, ctx = _shapes(c)
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    pt, n_slots = _pages(gen, ctx if c["kind"] != "gather" else ctx[:1], page, dev)
    kb, vb = _bank(gen, h_kv, d, dev, "k"), _bank(gen, h_kv, d, dev, "v")
    s = dict(kind=c["kind"], pt=pt, page=page, n_slots=n_slots, h_kv=h_kv, d=d)
    pick = torch.randint(0, 16384, (n_slots,), generator=gen, device=dev)
    if c["kind"] == "kv" or c["kind"] == "gather" or c["kind"] == "sparse" or c["fp4"]:
        (kc, ks), (vc, vs) = _quantise(kb, K_SCALE), _quantise(vb, V_SCALE)
        s.update(kc=kc[pick], ks=ks[pick], vc=vc[pick], vs=vs[pick])
    else:
        s.update(k=kb[pick], v=vb[pick])
    start = np.concatenate([[0], np.cumsum(n)])
    if c["kind"] == "kv":
        t = int(start[-1])
        at = torch.randint(0, 16384, (t,), generator=gen, device=dev)
        pos = np.concatenate([np.arange(f, f + m) for m, f in zip(n, first)])
        req = torch.as_tensor(np.repeat(np.arange(len(n)), n), device=dev)
        p = torch.as_tensor(pos, device=dev)
        slots = (pt[req, p // page].long() * page + p % page).to(torch.int32)
        s.update(k_new=kb[at], v_new=vb[at], start=i32(start), first=i32(first), slots=slots,
                 k_out=torch.empty((t, h_kv, d), dtype=torch.bfloat16, device=dev),
                 v_out=torch.empty((t, h_kv, d), dtype=torch.bfloat16, device=dev))
        return s
    if c["kind"] in ("gather", "sparse"):
        L = _rows(n, ctx) if c["kind"] == "sparse" else ctx
        req = np.repeat(np.arange(len(n)), n) if c["kind"] == "sparse" else np.zeros(len(ctx), np.int64)
        rows, w, run = len(L), c["n_idx"], c.get("run", 4)
        # a selection: runs of `run` consecutive positions, ascending, as many as the row has
        nb = -(-w // run)
        Lt, rq = torch.as_tensor(L, device=dev), torch.as_tensor(req, device=dev)
        blocks = (Lt // run).clamp(min=1)
        at = torch.linspace(0, 1, nb + 1, device=dev, dtype=torch.float64)[:nb]
        jit = torch.rand((rows, nb), generator=gen, device=dev, dtype=torch.float64) / (nb + 1)
        b = ((at[None] + jit) * blocks[:, None]).long().clamp(max=blocks[:, None] - 1)
        few = blocks[:, None] <= nb
        b = torch.where(few, torch.arange(nb, device=dev)[None].expand(rows, nb), b)
        p = (b[:, :, None] * run + torch.arange(run, device=dev)).flatten(1)[:, :w]
        slots = pt[rq[:, None], (p.clamp(max=int(max(ctx)) - 1) // page)].long() * page + p % page
        gone = p >= Lt[:, None]
        if c.get("holes"):
            gone = gone | (torch.rand((rows, w), generator=gen, device=dev) < c["holes"])
        s["slots"] = torch.where(gone, torch.full_like(slots, -1), slots).to(torch.int32).contiguous()
        if c["kind"] == "gather":
            s.update(k_out=torch.empty((rows, w, h_kv, d), dtype=torch.bfloat16, device=dev),
                     v_out=torch.empty((rows, w, h_kv, d), dtype=torch.bfloat16, device=dev))
            return s
    else:
        L = _rows(n, ctx)
        rows = len(L)
        req = torch.as_tensor(np.repeat(np.arange(len(n)), n), device=dev)
        s.update(fp4=c["fp4"], window=c["window"], n_sink=c["n_sink"], start=i32(start), row_len=i32(L), req=req,
                 max_len=int(max(ctx)), max_rows=int(max(n)), ctx=torch.as_tensor(ctx, device=dev))
    h_q = c["h_q"]
    s["q"] = torch.randn((rows, h_q, d), generator=gen, device=dev).to(torch.bfloat16)
    s["scale"] = d ** -0.5
    s["out"] = torch.empty((rows, h_q, d), dtype=torch.float32 if c["kind"] == "sparse" else torch.bfloat16, device=dev)
    s["lse"] = torch.empty((rows, h_q), dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------- runs
def _softmax_rows(logit, v, eq):
    """Attention weights of masked (-inf) logits times v; empty rows give 0 and -inf."""
    m = logit.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(logit - m)
    z = e.sum(-1, keepdim=True)
    o = torch.einsum(eq, torch.where(z > 0, e / z, torch.zeros_like(e)), v)
    return o, (m + torch.log(z))[..., 0]


def _plain_slots(s, g, codes, scales, slots):
    at = slots.long().clamp(min=0)
    return torch.where((slots >= 0)[..., None, None], _values(codes[at], scales[at], g), torch.zeros((), device=slots.device))


def _plain(s):
    k = s["kind"]
    if k == "kv":
        t = s["k_new"].shape[0]
        i = torch.arange(t, device=s["pt"].device)
        r = torch.searchsorted(s["start"][1:].contiguous(), i.to(torch.int32), right=True)
        p = s["first"][r] + i - s["start"][r]
        at = s["pt"][r, p // s["page"]].long() * s["page"] + p % s["page"]
        s["kc"][at], s["ks"][at] = _quantise(s["k_new"], K_SCALE)
        s["vc"][at], s["vs"][at] = _quantise(s["v_new"], V_SCALE)
    if k == "kv" or k == "gather":
        return (_plain_slots(s, K_SCALE, s["kc"], s["ks"], s["slots"]).to(torch.bfloat16),
                _plain_slots(s, V_SCALE, s["vc"], s["vs"], s["slots"]).to(torch.bfloat16))
    h_kv, d = s["h_kv"], s["d"]
    if k == "sparse":
        kk = _plain_slots(s, K_SCALE, s["kc"], s["ks"], s["slots"])
        vv = _plain_slots(s, V_SCALE, s["vc"], s["vs"], s["slots"])
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
    if s["fp4"]:
        kk = _plain_slots(s, K_SCALE, s["kc"], s["ks"], slots)
        vv = _plain_slots(s, V_SCALE, s["vc"], s["vs"], slots)
    else:
        kk, vv = s["k"][slots.clamp(min=0)].float(), s["v"][slots.clamp(min=0)].float()
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
    if k == "kv":
        qsa.append_kv_fp4(s["k_new"], s["v_new"], s["start"], s["first"], s["kc"], s["ks"], s["vc"], s["vs"], s["pt"],
                          s["page"], K_SCALE, V_SCALE)
    if k == "kv" or k == "gather":
        return qsa.gather_kv_fp4(s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], K_SCALE, V_SCALE, k_out=s["k_out"],
                                 v_out=s["v_out"])
    if k == "sparse":
        return qsa.sparse_attn_fp4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], s["scale"], K_SCALE, V_SCALE,
                                   out=s["out"], lse=s["lse"])
    if s["fp4"]:
        return qsa.window_attn_fp4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["start"], s["row_len"], s["pt"],
                                   s["page"], s["max_len"], s["window"], s["n_sink"], s["scale"], K_SCALE, V_SCALE,
                                   max_rows_per_req=s["max_rows"], out=s["out"], lse=s["lse"])
    return qsa.window_attn(s["q"], s["k"], s["v"], s["start"], s["row_len"], s["pt"], s["page"], s["max_len"],
                           s["window"], s["n_sink"], s["scale"], max_rows_per_req=s["max_rows"], out=s["out"],
                           lse=s["lse"])


# --------------------------------------------------------------------- exact
def _read64(codes, scales, g):
    """Values in FP64, decoded from the bits: e2m1 = (-1)^s (m + 2 [e > 0]) 2^(max(e, 1) - 2),
    e4m3 = (m + 8 [e > 0]) 2^(max(e, 1) - 10)."""
    c = codes.to(torch.int64)
    n = torch.stack((c % 16, c // 16), dim=-1).reshape(*codes.shape[:-1], -1)
    e, m = n // 2 % 4, n % 2
    v = (m + 2 * (e > 0)).double() * torch.pow(2.0, (e.clamp(min=1) - 2).double()) * (1 - 2 * (n // 8)).double()
    u = scales.to(torch.int64)
    e, m = u // 8 % 16, u % 8
    f = (m + 8 * (e > 0)).double() * torch.pow(2.0, (e.clamp(min=1) - 10).double()) * float(np.float32(g))
    return v * f.repeat_interleave(16, -1)


def _round64(x, g):
    """x after a round trip through the 4-bit blocks, in FP64."""
    g = float(np.float32(g))
    b = x.double().reshape(*x.shape[:-1], -1, 16)
    top = (b.abs().max(dim=-1).values / (6 * g)).clamp(max=448.0)
    step = torch.pow(2.0, torch.floor(torch.log2(top.clamp(min=2.0 ** -6))) - 3)
    f = (torch.round(top / step) * step).clamp(max=448.0)[..., None] * g  # torch.round: halves to even
    y = torch.where(f > 0, b / torch.where(f > 0, f, torch.ones_like(f)), torch.zeros_like(b))
    a = y.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(y) * torch.round(a / step) * step * f).reshape(x.shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "kv":
        return _round64(s["k_new"], K_SCALE), _round64(s["v_new"], V_SCALE)
    if c["kind"] == "gather":
        at = s["slots"].long()
        keep = (at >= 0).double()[..., None, None]
        at = at.clamp(min=0)
        return (_read64(s["kc"][at], s["ks"][at], K_SCALE) * keep, _read64(s["vc"][at], s["vs"][at], V_SCALE) * keep)
    n, _, ctx = _shapes(c)
    L, h_q, h_kv, d = _rows(n, ctx), c["h_q"], c["h_kv"], c["d"]
    grp, dev = h_q // h_kv, s["pt"].device
    out = torch.zeros((len(L), h_q, d), dtype=torch.float64, device=dev)
    lse = torch.full((len(L), h_q), -math.inf, dtype=torch.float64, device=dev)

    def attend(t0, t1, slots, seen):
        if c["kind"] == "sparse" or c["fp4"]:
            kk = _read64(s["kc"][slots], s["ks"][slots], K_SCALE)
            vv = _read64(s["vc"][slots], s["vs"][slots], V_SCALE)
        else:
            kk, vv = s["k"][slots].double(), s["v"][slots].double()
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
        slots = s["pt"][r].long()[pos // s["page"]] * s["page"] + pos % s["page"]
        Lr = torch.as_tensor(L[t0:t0 + m], device=dev)[:, None]
        attend(t0, t0 + m, slots, (pos < Lr) & ((pos >= Lr - c["window"]) | (pos < c["n_sink"])))
        t0 += m
    return out, lse
