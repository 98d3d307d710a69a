"""The paged key-value cache operators, as they are measured: block tables and slot maps from
request lengths, the store of new keys and values, and attention of new tokens over the cache.

A case is one call at fixed sizes. Request lengths are spread evenly over the logarithm of
their range and are the same for every seed, in an order that the seed draws, so the work of a
case is known from the case alone; values and page numbers come from the seed. `run` computes a
call in its plain form (elementary torch operations in fp32, rounded once) or, with `own` true,
through draft_candidate_selector_gb300. `exact` gives the same results in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0

# An attention case: R requests with n_lo..n_hi new tokens on ctx_lo..ctx_hi cached ones, Hq query
# and Hkv key heads of D values, pages of `page` tokens. left and right bound the keys a token sees
# (-1: no bound; right 0: causal).
_ATTEND = dict(op="attend", dtype="bf16", cache="bf16", layout="nhd", left=-1, right=0,
               softcap=0.0)


def listed():
    return [
        # One draft step's bookkeeping: 1 bonus + 15 mask tokens for each of 64 requests.
        dict(name="tables, draft step", op="tables", R=64, n_lo=16, n_hi=16, ctx_lo=100,
             ctx_hi=8000, page=16),
        # A batch of new prompts enters at once.
        dict(name="tables, new prompts", op="tables", R=700, n_lo=31, n_hi=2500, ctx_lo=0,
             ctx_hi=0, page=32),
        # The keys and values of one draft step, one layer.
        dict(name="store, draft step", op="store", T=1024, Hkv=8, D=128, page=16, dtype="bf16",
             cache="bf16", layout="nhd"),
        # Prompt chunks into an 8-bit cache.
        dict(name="store, prompts, 8-bit", op="store", T=40001, Hkv=8, D=128, page=64,
             dtype="bf16", cache="e4m3", layout="nhd"),
        # The smallest call: one user, one token, a short context.
        dict(_ATTEND, name="one token, short context", R=1, n_lo=1, n_hi=1, ctx_lo=332,
             ctx_hi=332, Hq=16, Hkv=8, D=128, page=16),
        # Plain decoding of a batch.
        dict(_ATTEND, name="single tokens, batch", R=96, n_lo=1, n_hi=1, ctx_lo=500,
             ctx_hi=16000, Hq=32, Hkv=8, D=128, page=16),
        # Plain decoding from an 8-bit cache.
        dict(_ATTEND, name="single tokens, 8-bit cache", R=128, n_lo=1, n_hi=1, ctx_lo=200,
             ctx_hi=20000, Hq=32, Hkv=4, D=128, page=64, cache="e4m3"),
        # One user, one token, a very long context.
        dict(_ATTEND, name="one token, long context", R=1, n_lo=1, n_hi=1, ctx_lo=200000,
             ctx_hi=200000, Hq=32, Hkv=8, D=128, page=32),
        # A target model verifies drafted blocks of 1 + 15 tokens.
        dict(_ATTEND, name="blocks, causal", R=64, n_lo=16, n_hi=16, ctx_lo=500, ctx_hi=8000,
             Hq=32, Hkv=8, D=128, page=16),
        # The block drafter's own attention: not causal, a sliding window, capped scores.
        dict(_ATTEND, name="blocks, window", R=256, n_lo=16, n_hi=16, ctx_lo=100, ctx_hi=9000,
             Hq=32, Hkv=16, D=64, page=32, dtype="fp16", cache="fp16", layout="hnd", left=1023,
             right=-1, softcap=50.0),
        # Prompt chunks that follow earlier ones.
        dict(_ATTEND, name="chunks over context", R=3, n_lo=1001, n_hi=2048, ctx_lo=2000,
             ctx_hi=14000, Hq=32, Hkv=8, D=128, page=64),
        # One whole prompt.
        dict(_ATTEND, name="whole prompt", R=1, n_lo=16001, n_hi=16001, ctx_lo=0, ctx_hi=0,
             Hq=16, Hkv=4, D=128, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "store", "one", "one", "block", "block", "prompt", "prompt"])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    if kind == "tables":
        new = rng.random() < 0.5
        R = _log(rng, 1, 1000)
        hi = min(_log(rng, 4, 2500), 350000 // R) if new else rng.randint(1, 33)
        return dict(op="tables", R=R, n_lo=1 if rng.random() < 0.5 else hi, n_hi=hi,
                    ctx_lo=0 if new else _log(rng, 1, 3000),
                    ctx_hi=0 if new else _log(rng, 3000, 20000), page=page)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    layout = rng.choice(["nhd", "hnd"])
    D = rng.choice([64, 128, 128])
    if kind == "store":
        return dict(op="store", T=_log(rng, 1, 40000), Hkv=rng.choice([1, 2, 3, 4, 8]), D=D,
                    page=page, dtype=dtype, cache=cache, layout=layout)
    Hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    case = dict(_ATTEND, Hq=Hkv * group, Hkv=Hkv, D=D, page=page, dtype=dtype, cache=cache,
                layout=layout)
    most = int(1.7e9) // (Hkv * D * 4)          # cached tokens of all requests together
    if kind == "one":
        R = _log(rng, 1, 96)
        hi = min(_log(rng, 20, 200000), most // R)
        case.update(R=R, n_lo=1, n_hi=1, ctx_lo=max(1, hi // rng.choice([1, 3, 20])), ctx_hi=hi)
    elif kind == "block":
        R = _log(rng, 1, 96)
        hi = min(_log(rng, 20, 60000), most // R)
        n = rng.randint(2, 33)
        case.update(R=R, n_lo=rng.choice([1, n]), n_hi=n,
                    ctx_lo=max(1, hi // rng.choice([1, 4, 30])), ctx_hi=hi,
                    right=rng.choice([0, -1]), left=rng.choice([-1, -1, _log(rng, 16, 4096)]),
                    softcap=rng.choice([0.0, 0.0, 30.0]))
    else:
        R = rng.randint(1, 4)
        n = _log(rng, 65, 12000) // R + 1
        ctx = rng.choice([0, _log(rng, 100, 8000)])
        while 4.0 * R * n * (ctx + n) * Hkv * group * D > 1e12:
            n -= n // 8
        case.update(R=R, n_lo=max(1, n // rng.choice([1, 2, 5])), n_hi=n, ctx_lo=ctx // 2,
                    ctx_hi=ctx, left=rng.choice([-1, -1, _log(rng, 64, 4096)]),
                    softcap=rng.choice([0.0, 0.0, 30.0]))
    return case


# ---------------------------------------------------------------- sizes of a case

def _spread(lo, hi, R, stride):
    """R whole numbers spread over the logarithm of [lo, hi], in a fixed mixed order."""
    if hi <= 0:
        return np.zeros(R, dtype=np.int64)
    lo = max(lo, 1)
    at = np.arange(R) / max(1, R - 1) if R > 1 else np.ones(1)
    v = np.rint(lo * (hi / lo) ** at).astype(np.int64)
    while math.gcd(stride, R) != 1:
        stride += 1
    return v[(np.arange(R) * stride) % R]


def _lengths(case):
    """(cached tokens, new tokens) of each request."""
    return (_spread(case["ctx_lo"], case["ctx_hi"], case["R"], 7),
            _spread(case["n_lo"], case["n_hi"], case["R"], 11))


def _pages(tokens, page):
    return -(-tokens // page)


def _visible(case, ctx, n):
    """(pairs of a new token and a key it sees, keys that any of them sees) for one request."""
    pos = ctx + np.arange(n)
    total = ctx + n
    lo = np.zeros(n, dtype=np.int64) if case["left"] < 0 else np.maximum(0, pos - case["left"])
    hi = (np.full(n, total) if case["right"] < 0
          else np.minimum(total, pos + case["right"] + 1))
    return int(np.maximum(hi - lo, 0).sum()), int(max(0, hi.max() - lo.min()))


def work(case):
    if case["op"] == "store":
        n = case["T"] * case["Hkv"] * case["D"] * 2
        size = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": n * (2 + size) + case["T"] * 8, "flops": 0}
    ctx, new = _lengths(case)
    if case["op"] == "tables":
        T, R = int(new.sum()), case["R"]
        fresh = int((_pages(ctx + new, case["page"]) - _pages(ctx, case["page"])).sum())
        # lengths and held pages in, starts, lengths and held pages out; the fresh pages; a
        # position and a 64-bit slot for each token
        return {"bytes": 24 * R + 8 * fresh + 12 * T, "flops": 0}
    T = int(new.sum())
    seen = [_visible(case, int(c), int(n)) for c, n in zip(ctx, new)]
    pairs, keys = sum(p for p, _ in seen), sum(k for _, k in seen)
    size = 1 if case["cache"] == "e4m3" else 2
    return {"bytes": 2 * keys * case["Hkv"] * case["D"] * size
            + T * case["Hq"] * (case["D"] * 4 + 4)
            + 4 * sum(_pages(k, case["page"]) for _, k in seen),
            "flops": 4 * pairs * case["Hq"] * case["D"]}


# ---------------------------------------------------------------- inputs

def _cache(pages, case, dev):
    """An empty cache [pages, page, Hkv, D], in memory by token or by head."""
    P, H, D = case["page"], case["Hkv"], case["D"]
    dt = DTYPES[case["cache"]]
    if case["layout"] == "hnd":
        return torch.zeros((pages, H, P, D), dtype=dt, device=dev).transpose(1, 2)
    return torch.zeros((pages, P, H, D), dtype=dt, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = np.random.default_rng(seed)
    if case["op"] == "store":
        T, H, D, page = case["T"], case["Hkv"], case["D"], case["page"]
        dt = DTYPES[case["dtype"]]
        # keys and values are slices of a fused projection's output, four query heads beside
        # each key head
        qkv = torch.randn((T, 6 * H, D), generator=g, device=dev).to(dt)
        pages = _pages(T, page) + 3
        slots = torch.randperm(pages, generator=g, device=dev).repeat_interleave(page) * page
        slots = (slots + torch.arange(page, device=dev).repeat(pages))[:T].contiguous()
        pad = torch.rand(T, generator=g, device=dev) < 0.01           # padded tokens
        pad[0] = False
        slots = torch.where(pad, torch.full_like(slots, -1), slots)
        return dict(case=case, key=qkv[:, 4 * H:5 * H], value=qkv[:, 5 * H:], slots=slots,
                    key_cache=_cache(pages, case, dev), value_cache=_cache(pages, case, dev),
                    k_scale=0.0625 if case["cache"] == "e4m3" else 1.0,
                    v_scale=0.03125 if case["cache"] == "e4m3" else 1.0)
    ctx, new = _lengths(case)
    order = host.permutation(case["R"])
    ctx, new = ctx[order], new[order]
    total = ctx + new
    page = case["page"]
    i32 = dict(dtype=torch.int32, device=dev)
    if case["op"] == "tables":
        held, need = _pages(ctx, page), _pages(total, page)
        pool = int(need.sum()) + 64
        perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        width = int(need.max()) + 2
        table = torch.full((case["R"], width), -1, **i32)
        col = torch.arange(width, device=dev)[None, :]
        heldt = torch.tensor(held, device=dev)[:, None]
        first = torch.tensor(np.cumsum(held) - held, device=dev)[:, None]
        table = torch.where(col < heldt, perm[(first + col).clamp(max=pool - 1)], table)
        return dict(case=case, context_lens=torch.tensor(ctx, **i32),
                    new_lens=torch.tensor(new, **i32), held=torch.tensor(held, **i32),
                    free_pages=perm[int(held.sum()):].contiguous(), block_table=table,
                    T=int(new.sum()))
    need = _pages(total, page)
    pool = int(need.sum()) + 5
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    width = int(need.max())
    col = torch.arange(width, device=dev)[None, :]
    first = torch.tensor(np.cumsum(need) - need, device=dev)[:, None]
    needt = torch.tensor(need, device=dev)[:, None]
    table = torch.where(col < needt, perm[(first + col).clamp(max=pool - 1)],
                        torch.zeros((), **i32))
    T, D = int(new.sum()), case["D"]
    dt = DTYPES[case["dtype"]]
    small = case["cache"] == "e4m3"
    k_scale, v_scale = (0.0625, 0.03125) if small else (1.0, 1.0)
    # a few strong channels in the keys, as trained ones have, so that some scores stand out
    gain = torch.exp(0.5 * torch.randn((case["Hkv"], D), generator=g, device=dev))
    caches = []
    for s, by in ((k_scale, gain), (v_scale, 1.0)):
        c = _cache(pool, case, dev)
        for at in range(0, pool, 4096):
            v = torch.randn((min(4096, pool - at), page, case["Hkv"], D), generator=g, device=dev)
            v = v * by / s
            c[at:at + 4096] = (v.clamp(-E4M3_MAX, E4M3_MAX) if small else v).to(c.dtype)
        caches.append(c)
    qkv = torch.randn((T, case["Hq"] + 2 * case["Hkv"], D), generator=g, device=dev).to(dt)
    return dict(case=case, query=qkv[:, :case["Hq"]], key_cache=caches[0],
                value_cache=caches[1], block_table=table,
                query_start=torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32),
                kv_lens=torch.tensor(total, **i32), k_scale=k_scale, v_scale=v_scale,
                n_max=int(new.max()), scale=1.0 / math.sqrt(D))


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"tables": _own_tables, "store": _own_store, "attend": _own_attend}[op](s)
    return {"tables": _plain_tables, "store": _plain_store, "attend": _plain_attend}[op](s)


def _own_tables(s):
    import draft_candidate_selector_gb300 as ds

    query_start, kv_lens, held, positions, slots, needed = ds.dflash_block_tables(
        s["context_lens"], s["new_lens"], s["held"], s["free_pages"], s["block_table"],
        s["case"]["page"], s["T"])
    return dict(block_table=s["block_table"], query_start=query_start, kv_lens=kv_lens, held=held,
                positions=positions, slots=slots, needed=needed)


def _plain_tables(s):
    page, T = s["case"]["page"], s["T"]
    ctx, new, held = s["context_lens"], s["new_lens"], s["held"]
    R, table, free = ctx.numel(), s["block_table"], s["free_pages"]
    dev = ctx.device
    kv_lens = ctx + new
    need = (torch.div(kv_lens + page - 1, page, rounding_mode="floor") - held).clamp(min=0)
    start = torch.cumsum(need, 0) - need
    query_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev),
                             torch.cumsum(new, 0)]).to(torch.int32)
    col = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    src = (start[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[src], table))
    req = torch.repeat_interleave(torch.arange(R, device=dev), new.long(), output_size=T)
    positions = ctx[req] + (torch.arange(T, device=dev) - query_start[req])
    positions = positions.to(torch.int32)
    page_of = table[req, torch.div(positions, page, rounding_mode="floor").long()].long()
    return dict(block_table=table, query_start=query_start, kv_lens=kv_lens, held=held + need,
                positions=positions, slots=page_of * page + positions % page,
                needed=need.sum(dtype=torch.int32).reshape(1))


def _own_store(s):
    import draft_candidate_selector_gb300 as ds

    ds.dflash_store_kv(s["key"], s["value"], s["slots"], s["key_cache"], s["value_cache"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])
    return dict(key_cache=s["key_cache"], value_cache=s["value_cache"])


def _plain_put(x, slots, cache, scale, page):
    if cache.dtype == torch.float8_e4m3fn:
        x = (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        x, cache = x.view(torch.uint8), cache.view(torch.uint8)
    at = slots.clamp(min=0)
    block, row = torch.div(at, page, rounding_mode="floor"), at % page
    keep = (slots >= 0)[:, None, None]
    # a padded token (slot -1) puts back what the last slot in use holds or gets
    last = torch.argmax(slots)
    block, row = (torch.where(slots >= 0, v, v[last]) for v in (block, row))
    cache[block, row] = torch.where(keep, x, x[last][None])


def _plain_store(s):
    page = s["case"]["page"]
    _plain_put(s["key"], s["slots"], s["key_cache"], s["k_scale"], page)
    _plain_put(s["value"], s["slots"], s["value_cache"], s["v_scale"], page)
    return dict(key_cache=s["key_cache"], value_cache=s["value_cache"])


def _own_attend(s):
    import draft_candidate_selector_gb300 as ds

    c = s["case"]
    out, lse = ds.dflash_paged_attention(
        s["query"], s["key_cache"], s["value_cache"], s["block_table"], s["query_start"],
        s["kv_lens"], scale=s["scale"], window_left=c["left"], window_right=c["right"],
        softcap=c["softcap"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return dict(out=out, lse=lse)


def _plain_attend(s):
    c = s["case"]
    q, table, qs, kv = s["query"], s["block_table"], s["query_start"].long(), s["kv_lens"].long()
    T, Hq, D = q.shape
    Hkv, n, dev = c["Hkv"], s["n_max"], q.device
    R, L = kv.numel(), table.shape[1] * c["page"]
    i = torch.arange(n, device=dev)
    count = qs[1:] - qs[:-1]
    live = i[None, :] < count[:, None]                                    # [R, n]
    token = (qs[:-1, None] + i[None, :]).clamp(max=T - 1)
    qf = q[token].float().reshape(R, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    qf = qf.reshape(R, Hkv, -1, D)                                        # [R, Hkv, g n, D]
    at = table.long()
    as_rows = lambda x: (x.view(torch.uint8)[at].view(x.dtype)            # noqa: E731
                         if x.dtype == torch.float8_e4m3fn else x[at])
    k = as_rows(s["key_cache"]).float().reshape(R, L, Hkv, D).permute(0, 2, 3, 1)
    x = torch.matmul(qf, k) * (s["scale"] * s["k_scale"])                 # [R, Hkv, g n, L]
    del k
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    pos = kv[:, None] - count[:, None] + i[None, :]                       # [R, n]
    j = torch.arange(L, device=dev)
    seen = (j < kv[:, None, None]) & live[:, :, None]
    if c["right"] >= 0:
        seen = seen & (j <= pos[:, :, None] + c["right"])
    if c["left"] >= 0:
        seen = seen & (j >= pos[:, :, None] - c["left"])
    x = x.reshape(R, Hkv, -1, n, L).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = as_rows(s["value_cache"]).float().reshape(R, L, Hkv, D).permute(0, 2, 1, 3)
    o = torch.matmul(p.reshape(R, Hkv, -1, L), v).reshape(R, Hkv, -1, n, D)
    o = o * s["v_scale"] / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + torch.log(total)).squeeze(-1)                              # -inf where none is seen
    req = torch.repeat_interleave(torch.arange(R, device=dev), count, output_size=T)
    idx = torch.arange(T, device=dev) - qs[req]
    out = o.permute(0, 3, 1, 2, 4).reshape(R, n, Hq, D)[req, idx].to(q.dtype)
    return dict(out=out, lse=lse.permute(0, 3, 1, 2).reshape(R, n, Hq)[req, idx])


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    page = case["page"]
    if case["op"] == "store":
        got = {}
        for name, scale in (("key", s["k_scale"]), ("value", s["v_scale"])):
            c = s[name + "_cache"]
            full = torch.zeros(c.shape, dtype=torch.float64, device=c.device)
            x = s[name].double()
            if case["cache"] == "e4m3":
                x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)
            for t0 in range(0, case["T"], 8192):
                sl = s["slots"][t0:t0 + 8192]
                ok = sl >= 0
                full[sl[ok] // page, sl[ok] % page] = x[t0:t0 + 8192][ok]
            got[name + "_cache"] = full
        return got
    q, kv, qs = s["query"], s["kv_lens"].tolist(), s["query_start"].tolist()
    T, Hq, D = q.shape
    g = Hq // case["Hkv"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    for r in range(case["R"]):
        t0, t1, L = qs[r], qs[r + 1], kv[r]
        rows = s["block_table"][r, :_pages(L, page)].long()
        kr = s["key_cache"][rows].double() if case["cache"] != "e4m3" else \
            s["key_cache"].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double()
        vr = s["value_cache"][rows].double() if case["cache"] != "e4m3" else \
            s["value_cache"].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double()
        kr = kr.reshape(-1, case["Hkv"], D)[:L] * s["k_scale"]
        vr = vr.reshape(-1, case["Hkv"], D)[:L] * s["v_scale"]
        key_at = torch.arange(L, device=q.device)[None, :]
        for a in range(t0, t1, 4096):
            b = min(a + 4096, t1)
            where = torch.arange(L - (t1 - a), L - (t1 - b), device=q.device)[:, None]
            hidden = torch.zeros((b - a, L), dtype=torch.bool, device=q.device)
            if case["right"] >= 0:
                hidden |= key_at > where + case["right"]
            if case["left"] >= 0:
                hidden |= key_at < where - case["left"]
            for h in range(Hq):
                z = q[a:b, h].double() @ kr[:, h // g].T * s["scale"]
                if case["softcap"] > 0:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                z.masked_fill_(hidden, -math.inf)
                lse[a:b, h] = torch.logsumexp(z, 1)
                out[a:b, h] = torch.softmax(z, 1) @ vr[:, h // g]
    return dict(out=out, lse=lse)
