"""The operators around the paged attention and the selector in a sampled speculative step, as they
are measured: the norm and rotation of queries and keys (alone, or storing keys and values in the
paged cache in the same pass), a path drawn through the selector's edge scores, and the verification
of drafted tokens against the target's logits.

A case is one call at fixed sizes. Lengths, and how many drafts of each request are accepted, are
spread evenly over their range and are the same for every seed, in an order that the seed draws, so
the work of a case is known from the case alone; values come from the seed. `run` computes a call in
its plain form (elementary torch operations) or, with `own` true, through
draft_candidate_selector_gb300. `exact` gives the same results in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0

# Norm and rotation of T tokens' Hq query and Hkv key heads of D values at positions up to `far`.
# cache: None, or the type of a paged cache that takes the keys and values. rotary: values of a head
# that are rotated. factor, original: positions past `original` tokens by a longer wave of the slow pairs.
_ROPE = dict(op="rope", dtype="bf16", cache=None, page=16, rotary=128, interleaved=False, norm=True,
             far=8000, factor=1.0, original=0)

# Verification of the drafts of R requests, each d_lo..d_hi tokens and at most S, against logits of V
# tokens in rows of V + pad_v. K: candidates that the draft's distribution spreads over (1: it is
# certain of its token). rate: chance that a draft is accepted. t_lo..t_hi: temperatures (0: greedy).
_VERIFY = dict(op="verify", dtype="bf16", S=15, d_lo=15, d_hi=15, K=8, rate=0.8, t_lo=1.0, t_hi=1.0,
               pad_v=0, pad_t=0)


def listed():
    return [
        # Plain decoding, one user: the smallest call.
        dict(_ROPE, name="norm and rotation, one token", T=1, Hq=16, Hkv=8, D=128),
        # One draft step of 64 requests, 1 bonus + 15 mask tokens each, into the cache.
        dict(_ROPE, name="norm, rotation, store: draft step", T=1024, Hq=32, Hkv=8, D=128, cache="bf16"),
        # New prompts into an 8-bit cache.
        dict(_ROPE, name="norm, rotation, store: prompts, 8-bit", T=40001, Hq=32, Hkv=8, D=128,
             cache="e4m3", page=64, far=20000),
        # Neighbouring pairs of half of each head, no norm, a context stretched sixteen times.
        dict(_ROPE, name="rotation, half a head, far positions", T=16411, Hq=32, Hkv=16, D=64,
             dtype="fp16", rotary=32, interleaved=True, norm=False, far=1000000, factor=16.0,
             original=65536),
        # The selector's own smallest sizes, then those of its larger workloads.
        dict(op="path", name="path, two requests", R=2, S=4, K=4, t_lo=1.0, t_hi=1.0),
        dict(op="path", name="path, batch", R=64, S=15, K=8, t_lo=0.6, t_hi=1.4),
        dict(op="path", name="path, large batch", R=512, S=15, K=32, t_lo=1.0, t_hi=1.0),
        # One user, a block of seven drafts.
        dict(_VERIFY, name="verify, one user", R=1, S=7, d_lo=7, d_hi=7, V=32768),
        # A batch of blocks whose drafts were drawn from the selector's edges.
        dict(_VERIFY, name="verify, batch", R=64, V=151936),
        # Blocks of every length, none among them, odd rows, a temperature for each request.
        dict(_VERIFY, name="verify, ragged", R=37, S=12, d_lo=0, d_hi=12, V=100003, pad_v=93, pad_t=5,
             dtype="fp16", K=5, t_lo=0.6, t_hi=1.4),
        # Greedy target, certain drafts, a large batch.
        dict(_VERIFY, name="verify, greedy", R=512, V=151936, K=1, rate=0.85, t_lo=0.0, t_hi=0.0),
        # The largest: logits in 32 bits, the largest vocabulary.
        dict(_VERIFY, name="verify, large batch, 32 bits", R=256, V=262144, K=16, dtype="fp32",
             rate=0.85),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "rope", "path", "verify", "verify", "verify"])
    t_lo, t_hi = rng.choice([(1.0, 1.0), (1.0, 1.0), (0.5, 1.5), (0.3, 0.9)])
    if kind == "path":
        return dict(op="path", R=_log(rng, 1, 512), S=rng.randint(1, 15), K=rng.randint(1, 32),
                    t_lo=t_lo, t_hi=t_hi)
    if kind == "verify":
        V = _log(rng, 1000, 262144)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        S = rng.randint(0, 15)
        R = min(_log(rng, 1, 512), max(1, int(1e9) // (V * (S + 1))))
        if rng.random() < 0.2:
            t_lo = t_hi = 0.0
        return dict(_VERIFY, R=R, S=S, d_lo=rng.choice([S, S, 0]), d_hi=S, V=V, dtype=dtype,
                    K=rng.choice([1, 1, rng.randint(2, 32), 8, 16]), rate=rng.uniform(0.4, 0.95),
                    t_lo=t_lo, t_hi=t_hi, pad_v=rng.choice([0, 0, 0, rng.randint(1, 300)]),
                    pad_t=rng.choice([0, 0, rng.randint(1, 40)]))
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    case = dict(_ROPE, Hq=Hkv * rng.choice([1, 2, 3, 4, 4, 7, 8]), Hkv=Hkv, D=D,
                page=rng.choice([8, 16, 16, 32, 64, 24]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                rotary=rng.choice([D, D, D, D // 2, D // 4]), interleaved=rng.random() < 0.4,
                norm=rng.random() < 0.75, far=_log(rng, 1000, 2000000))
    if rng.random() < 0.3:
        case.update(factor=float(rng.randint(2, 40)), original=rng.choice([0, 4096, 32768]))
    if rng.random() < 0.6:
        case["cache"] = rng.choice([case["dtype"], case["dtype"], "e4m3"])
    most = int(2.4e8) // ((case["Hq"] + 2 * Hkv) * D)
    case["T"] = _log(rng, 1, min(40000, most))
    return case


# ---------------------------------------------------------------- sizes of a case

def _drafts(case):
    """(drafts, accepted drafts) of each request, in a fixed mixed order: drafts spread over their
    range, accepted ones as runs of successes of chance `rate` are."""
    R = case["R"]
    i = np.arange(R)
    d = np.rint(case["d_lo"] + (case["d_hi"] - case["d_lo"]) * i / max(1, R - 1)).astype(np.int64)
    stride = 7
    while math.gcd(stride, R) != 1:
        stride += 1
    run = np.floor(np.log(1 - ((i * stride) % R + 0.5) / R) / math.log(case["rate"])).astype(np.int64)
    return d, np.minimum(run, d)


def work(case):
    if case["op"] == "rope":
        T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
        size = SIZES[case["dtype"]]
        if case["cache"] is None:
            nbytes = 2 * T * (Hq + Hkv) * D * size + 4 * T
        else:
            nbytes = (2 * T * Hq * D * size + 2 * T * Hkv * D * (size + SIZES[case["cache"]])
                      + 12 * T)
        return {"bytes": nbytes, "flops": T * (Hq + Hkv) * (D * (4 if case["norm"] else 0)
                                                           + 3 * case["rotary"])}
    if case["op"] == "path":
        R, S, K = case["R"], case["S"], case["K"]
        # the row of edges behind each chosen token, a number and a token; a place, a token and K
        # probabilities out
        return {"bytes": 4 * R * S * (2 * K + 4), "flops": 4 * R * S * K}
    d, a = _drafts(case)
    # the rows up to the first rejected draft, or the last; the drafts that these rows look at
    rows, looked = int((a + 1).sum()), int(np.minimum(a + 1, d).sum())
    q = 8 * case["K"] if case["K"] > 1 and case["t_hi"] > 0 else 0
    return {"bytes": rows * case["V"] * SIZES[case["dtype"]] + looked * (8 + q)
            + 4 * case["R"] * (2 * case["S"] + 5),
            "flops": 4 * rows * case["V"]}


# ---------------------------------------------------------------- inputs

def _inverse_frequencies(case):
    """Radians a position of each pair: base 10000; pairs that turn less than once over `original`
    tokens are slowed `factor` times, those that turn 32 times or more are not, the others in between."""
    j = np.arange(case["rotary"] // 2)
    f = 10000.0 ** (-2.0 * j / case["rotary"])
    if case["factor"] != 1.0:
        if case["original"]:
            turns = case["original"] * f / (2 * math.pi)
            keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
        else:
            keep = np.zeros_like(f)
        f = f / case["factor"] * (1 - keep) + f * keep
    return f


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0


def _prepare_rope(case, g, dev):
    T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
    dt = DTYPES[case["dtype"]]
    gain = torch.exp(0.5 * torch.randn((Hq + 2 * Hkv, D), generator=g, device=dev))
    qkv = torch.empty((T, Hq + 2 * Hkv, D), dtype=dt, device=dev)
    for at in range(0, T, 4096):
        part = qkv[at:at + 4096]
        part.copy_(torch.randn(part.shape, generator=g, device=dev) * gain)
    # tokens of requests, each a run of positions
    first = torch.randint(0, case["far"], (T,), generator=g, device=dev)
    i = torch.arange(T, device=dev)
    positions = (first[i - i % 16] + i % 16).to(torch.int32)
    s = dict(case=case, query=qkv[:, :Hq], key=qkv[:, Hq:Hq + Hkv], value=qkv[:, Hq + Hkv:],
             positions=positions, q_weight=None, k_weight=None,
             inv_freq=torch.tensor(_inverse_frequencies(case), device=dev),
             magnitude=_magnitude(case))
    if case["norm"]:
        s["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
    if own:
        import draft_candidate_selector_gb300 as ds

        s["frequencies"] = ds.dflash_rope_frequencies(
            case["rotary"], factor=case["factor"], original_len=case["original"], device=dev)
    if case["cache"] is not None:
        page = case["page"]
        pages = -(-T // page) + 3
        slots = torch.randperm(pages, generator=g, device=dev).repeat_interleave(page) * page
        s["slots"] = (slots + torch.arange(page, device=dev).repeat(pages))[:T].contiguous()
        ct = DTYPES[case["cache"]]
        s["key_cache"] = torch.zeros((pages, page, Hkv, D), dtype=ct, device=dev)
        s["value_cache"] = torch.zeros_like(s["key_cache"])
        small = case["cache"] == "e4m3"
        s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if small else (1.0, 1.0)
    return s


def _temperatures(case, g, dev):
    """One for all requests, or one for each."""
    if case["t_lo"] == case["t_hi"]:
        return case["t_lo"]
    t = torch.rand(case["R"], generator=g, device=dev)
    return case["t_lo"] + (case["t_hi"] - case["t_lo"]) * t


def _prepare_path(case, g, dev):
    R, S, K = case["R"], case["S"], case["K"]
    # candidates in the order of their logits, and how well each follows the one before it
    unary = torch.randn((R, S, K), generator=g, device=dev).sort(-1, descending=True).values
    edges = 8 + 2 * unary[:, :, None] + torch.randn((R, S, K, K), generator=g, device=dev)
    edges[:, 0] = edges[:, 0, :1]
    ids = torch.randint(0, 262144 // K, (R, S, K), generator=g, device=dev) * K
    ids = (ids + torch.arange(K, device=dev)).to(torch.int32)
    return dict(case=case, edges=edges.contiguous(), cand_ids=ids,
                uniforms=torch.rand((R, S), generator=g, device=dev),
                temperature=_temperatures(case, g, dev))


def _prepare_verify(case, g, dev, host):
    R, S, V, K = case["R"], case["S"], case["V"], case["K"]
    d, a = _drafts(case)
    order = host.permutation(R)
    d, a = d[order], a[order]
    start = np.concatenate([[0], np.cumsum(d + 1)])
    T = int(start[-1]) + case["pad_t"]
    dt = DTYPES[case["dtype"]]
    logits = torch.zeros((T, V + case["pad_v"]), dtype=dt, device=dev)[:, :V]
    t = _temperatures(case, g, dev)
    greedy = isinstance(t, float) and t == 0.0
    temps = (torch.full((R,), t, device=dev) if isinstance(t, float) else t)
    wide = max(K, 4)                                             # likely tokens of each row
    dt_ = torch.tensor(d, device=dev)
    at_ = torch.tensor(a, device=dev)
    st_ = torch.tensor(start[:-1], device=dev)
    tokens = torch.zeros((R, S), dtype=torch.int32, device=dev)
    ids = torch.zeros((R, S, K), dtype=torch.int32, device=dev)
    probs = torch.zeros((R, S, K), device=dev)
    uniforms = torch.rand((R, S), generator=g, device=dev)
    for i in range(S + 1):
        x = 2 * torch.randn((R, V), generator=g, device=dev)
        cand = torch.randint(0, V // wide, (R, wide), generator=g, device=dev) * wide
        cand = cand + torch.arange(wide, device=dev)
        # the likely tokens hold most of a row's probability, some rows more of it than others
        lift = (math.log(V) + 2 + 4 * torch.rand((R, 1), generator=g, device=dev)
                + torch.randn((R, wide), generator=g, device=dev))
        x.scatter_(1, cand, lift)
        x = x.to(dt)
        live = (dt_ >= i).nonzero()[:, 0]
        logits[st_[live] + i] = x[live]
        if i == S:
            break
        xf = x.float()
        if greedy:
            top = xf.argmax(1)
            tokens[:, i] = torch.where(at_ > i, top, (top + 1) % V).to(torch.int32)
            ids[:, i] = tokens[:, i, None]
            probs[:, i] = 1.0 / K
            continue
        z = xf.div_(temps[:, None])
        lz = z.logsumexp(1, keepdim=True)
        likely = (z.gather(1, cand) - lz).exp()                  # the target's p of them
        cand_k, pk = cand[:, :K], likely[:, :K]
        if K == 1:
            q = torch.ones_like(pk)
            pick = torch.zeros((R, 1), dtype=torch.int64, device=dev)
        else:
            noise = 0.7 * torch.randn((R, K), generator=g, device=dev)
            q = torch.softmax(pk.log() + noise, 1)
            drawn = torch.multinomial(q, 1, generator=g)
            worst = (pk / q).argmin(1, keepdim=True)
            pick = torch.where((at_ > i)[:, None], drawn, worst)
        ratio = (pk.gather(1, pick) / q.gather(1, pick))[:, 0].clamp(max=1.0)
        u = uniforms[:, i]
        uniforms[:, i] = torch.where(at_ > i, u * ratio, ratio + (1 - ratio) * u).clamp(max=1 - 2 ** -24)
        tokens[:, i] = cand_k.gather(1, pick)[:, 0].to(torch.int32)
        ids[:, i] = cand_k.to(torch.int32)
        probs[:, i] = q
    return dict(case=case, logits=logits, draft_tokens=tokens,
                query_start=torch.tensor(start, dtype=torch.int32, device=dev),
                cand_ids=ids if K > 1 else None, draft_probs=probs if K > 1 else None,
                accept_uniforms=uniforms, sample_uniforms=torch.rand(R, generator=g, device=dev),
                temperature=t)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, g, dev)
    if case["op"] == "path":
        return _prepare_path(case, g, dev)
    return _prepare_verify(case, g, dev, np.random.default_rng(seed))


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "path": _own_path, "verify": _own_verify}[op](s)
    return {"rope": _plain_rope, "path": _plain_path, "verify": _plain_verify}[op](s)


def _own_rope(s):
    import draft_candidate_selector_gb300 as ds

    c = s["case"]
    how = dict(frequencies=s["frequencies"], q_weight=s["q_weight"], k_weight=s["k_weight"],
               interleaved=c["interleaved"], rope_scale=s["magnitude"])
    if c["cache"] is None:
        query, key = ds.dflash_qk_norm_rope(s["query"], s["key"], s["positions"], **how)
        return dict(query=query, key=key)
    query, key_cache, value_cache = ds.dflash_qk_norm_rope_store(
        s["query"], s["key"], s["value"], s["positions"], s["slots"], s["key_cache"],
        s["value_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"], **how)
    return dict(query=query, key_cache=key_cache, value_cache=value_cache)


def _plain_rotated(x, weight, cos, sin, c):
    """fp32 [T, heads, D]: normed, then the first `rotary` values of each head rotated."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    n = c["rotary"]
    if c["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_put(x, scale, slots, cache):
    page = cache.shape[1]
    if cache.dtype == torch.float8_e4m3fn:
        x = (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        x, cache = x.view(torch.uint8), cache.view(torch.uint8)
    cache[torch.div(slots, page, rounding_mode="floor"), slots % page] = x.to(cache.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]       # far positions: 64 bits
    cos = (angle.cos() * s["magnitude"]).float()
    sin = (angle.sin() * s["magnitude"]).float()
    query = _plain_rotated(s["query"], s["q_weight"], cos, sin, c).to(s["query"].dtype)
    key = _plain_rotated(s["key"], s["k_weight"], cos, sin, c)
    if c["cache"] is None:
        return dict(query=query, key=key.to(s["key"].dtype))
    _plain_put(key, s["k_scale"], s["slots"], s["key_cache"])
    _plain_put(s["value"], s["v_scale"], s["slots"], s["value_cache"])
    return dict(query=query, key_cache=s["key_cache"], value_cache=s["value_cache"])


def _own_path(s):
    import draft_candidate_selector_gb300 as ds

    path, tokens, probs = ds.dflash_sample_path(s["edges"], s["cand_ids"], s["uniforms"],
                                                temperature=s["temperature"])
    return dict(path=path, tokens=tokens, probs=probs)


def _plain_path(s):
    # 64 bits: a running sum is compared with a border
    E, u, t = s["edges"].double(), s["uniforms"].double(), s["temperature"]
    if not isinstance(t, float):
        t = t.double()[:, None]
    R, S, K, _ = E.shape
    prev = torch.zeros((R, 1, 1), dtype=torch.int64, device=E.device)
    path, probs = [], []
    for p in range(S):
        row = E[:, p].gather(1, prev.expand(R, 1, K))[:, 0]
        w = torch.exp((row - row.amax(1, keepdim=True)) / t)
        run_sum = w.cumsum(1)
        total = run_sum[:, -1:]
        pick = (run_sum <= u[:, p, None] * total).sum(1).clamp(max=K - 1)
        path.append(pick)
        probs.append((w / total).float())
        prev = pick[:, None, None]
    path = torch.stack(path, 1)
    return dict(path=path.to(torch.int32), tokens=s["cand_ids"].gather(2, path[:, :, None])[:, :, 0],
                probs=torch.stack(probs, 1))


def _own_verify(s):
    import draft_candidate_selector_gb300 as ds

    tokens, counts, logprobs = ds.dflash_verify_drafts(
        s["logits"], s["query_start"], s["draft_tokens"], s["accept_uniforms"], s["sample_uniforms"],
        cand_ids=s["cand_ids"], draft_probs=s["draft_probs"], temperature=s["temperature"])
    return dict(tokens=tokens, counts=counts, logprobs=logprobs)


def _plain_target(x, t):
    """The target's probabilities of rows x [R, V] at temperatures t [R, 1], in 64 bits."""
    z = x.double()
    top = z.amax(1, keepdim=True)
    z = z.sub_(top)
    V = z.shape[1]
    index = torch.arange(V, device=z.device)
    first = torch.where(z == 0, index, V).amin(1, keepdim=True)  # greedy: the first of the largest
    greedy = (t == 0)
    z = z.div_(torch.where(greedy, torch.ones_like(t), t)).exp_()
    z = torch.where(greedy, (index == first).to(z.dtype), z)
    return z.div_(z.sum(1, keepdim=True))


def _plain_verify(s):
    logits, start = s["logits"], s["query_start"].long()
    R, S = s["draft_tokens"].shape
    dev = logits.device
    drafts = start[1:] - start[:-1] - 1
    t = s["temperature"]
    t = (torch.full((R, 1), t, dtype=torch.float64, device=dev) if isinstance(t, float)
         else t.double()[:, None])
    ids, probs = s["cand_ids"], s["draft_probs"]
    if ids is None:
        ids, probs = s["draft_tokens"][:, :, None], torch.ones((R, S, 1), device=dev)
    ids, probs = ids.long(), probs.double()
    x = s["draft_tokens"].long()
    stop = drafts.clone()                                        # the row that a token is drawn from
    logprobs = torch.zeros((R, S + 1), dtype=torch.float64, device=dev)
    for i in range(S - 1, -1, -1):
        p = _plain_target(logits[(start[:-1] + i).clamp(max=logits.shape[0] - 1)], t)
        px = p.gather(1, x[:, i, None])[:, 0]
        qx = (probs[:, i] * (ids[:, i] == x[:, i, None])).sum(1)
        logprobs[:, i] = px.log()
        rejected = ~(s["accept_uniforms"][:, i].double() * qx < px) & (i < drafts)
        stop = torch.where(rejected, torch.full_like(stop, i), stop)
    p = target = _plain_target(logits[start[:-1] + stop], t)
    if S > 0:
        at = stop.clamp(max=S - 1)[:, None, None].expand(R, 1, ids.shape[2])
        q = torch.zeros_like(p).scatter_add_(1, ids.gather(1, at)[:, 0], probs.gather(1, at)[:, 0])
        rest = (p - q).clamp(min=0)
        use = (stop < drafts)[:, None] & (rest.sum(1, keepdim=True) > 0)
        p = torch.where(use, rest, p)
    run_sum = p.cumsum(1)
    border = s["sample_uniforms"].double()[:, None] * run_sum[:, -1:]
    drawn = (run_sum <= border).sum(1).clamp(max=p.shape[1] - 1)
    col = torch.arange(S + 1, device=dev)[None, :]
    tokens = torch.cat([x, torch.zeros((R, 1), dtype=torch.int64, device=dev)], 1)
    tokens = torch.where(col == stop[:, None], drawn[:, None], tokens)
    tokens = torch.where(col > stop[:, None], torch.full_like(tokens, -1), tokens)
    last = target.gather(1, drawn[:, None]).log()
    logprobs = torch.where(col == stop[:, None], last, logprobs)
    logprobs = torch.where(col > stop[:, None], torch.zeros_like(logprobs), logprobs)
    return dict(tokens=tokens.to(torch.int32), counts=(stop + 1).to(torch.int32),
                logprobs=logprobs.float())


# ---------------------------------------------------------------- 64 bits

def _exact_heads(x, weight, s):
    """Normed and rotated [T, heads, D] in 64 bits, by complex numbers of modulus `magnitude`."""
    n, T = s["case"]["rotary"], x.shape[0]
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * weight.double()
    turn = torch.polar(torch.full((T, n // 2), s["magnitude"], dtype=torch.float64, device=x.device),
                       s["positions"].double()[:, None] * s["inv_freq"][None, :])[:, None]
    y = x.clone()
    if s["case"]["interleaved"]:
        pairs = torch.view_as_complex(x[..., :n].reshape(T, -1, n // 2, 2).contiguous())
        y[..., :n] = torch.view_as_real(pairs * turn).reshape(T, -1, n)
    else:
        z = torch.complex(x[..., :n // 2].contiguous(), x[..., n // 2:n].contiguous()) * turn
        y[..., :n // 2], y[..., n // 2:n] = z.real, z.imag
    return y


def _exact_cache(x, scale, s, cache):
    full = torch.zeros(cache.shape, dtype=torch.float64, device=cache.device)
    if s["case"]["cache"] == "e4m3":
        x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)
    full.flatten(0, 1)[s["slots"]] = x
    return full


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        query = _exact_heads(s["query"], s["q_weight"], s)
        key = _exact_heads(s["key"], s["k_weight"], s)
        if case["cache"] is None:
            return dict(query=query, key=key)
        return dict(query=query, key_cache=_exact_cache(key, s["k_scale"], s, s["key_cache"]),
                    value_cache=_exact_cache(s["value"].double(), s["v_scale"], s, s["value_cache"]))
    t = s["temperature"]
    temps = [t] * case["R"] if isinstance(t, float) else t.double().tolist()
    if case["op"] == "path":
        E, u = s["edges"].double().cpu().numpy(), s["uniforms"].double().cpu().numpy()
        ids = s["cand_ids"].cpu().numpy()
        R, S, K, _ = E.shape
        path, probs = np.zeros((R, S), np.int32), np.zeros((R, S, K))
        for r in range(R):
            before = 0
            for i in range(S):
                w = np.exp((E[r, i, before] - E[r, i, before].max()) / temps[r])
                probs[r, i] = w / math.fsum(w)
                border, so_far, before = u[r, i] * math.fsum(w), 0.0, K - 1
                for c in range(K):
                    so_far += w[c]
                    if so_far > border:
                        before = c
                        break
                path[r, i] = before
        tokens = np.take_along_axis(ids, path[:, :, None].astype(np.int64), 2)[:, :, 0]
        out = dict(path=path, tokens=tokens, probs=probs)
        return {k: torch.tensor(v, device="cuda") for k, v in out.items()}
    logits, start = s["logits"], s["query_start"].tolist()
    drafted, u = s["draft_tokens"].tolist(), s["accept_uniforms"].double().tolist()
    last = s["sample_uniforms"].double().tolist()
    tokens, counts, logprobs = [], [], []
    for r in range(case["R"]):
        n, got, lp = start[r + 1] - start[r], [], []
        for i in range(n):
            z = logits[start[r] + i].double()
            if temps[r] == 0:
                p = torch.zeros_like(z)
                p[int((z == z.max()).nonzero()[0])] = 1.0
            else:
                p = torch.softmax(z / temps[r], 0)
            target = p
            if i < n - 1:
                q = torch.zeros_like(p)
                if s["cand_ids"] is None:
                    q[drafted[r][i]] = 1.0
                else:
                    for c, v in zip(s["cand_ids"][r, i].tolist(), s["draft_probs"][r, i].tolist()):
                        q[c] += v
                if u[r][i] * float(q[drafted[r][i]]) < float(p[drafted[r][i]]):
                    got.append(drafted[r][i])
                    lp.append(math.log(float(target[got[-1]])))
                    continue
                rest = torch.clamp(p - q, min=0)
                if float(rest.sum()) > 0:
                    p = rest
            so_far = torch.cumsum(p, 0)
            above = so_far > last[r] * so_far[-1]
            got.append(int(above.to(torch.uint8).argmax()) if bool(above.any()) else case["V"] - 1)
            lp.append(math.log(float(target[got[-1]])))
            break
        counts.append(len(got))
        logprobs.append(lp + [0.0] * (case["S"] + 1 - len(lp)))
        tokens.append(got + [-1] * (case["S"] + 1 - len(got)))
    return dict(tokens=torch.tensor(tokens, dtype=torch.int32, device="cuda"),
                counts=torch.tensor(counts, dtype=torch.int32, device="cuda"),
                logprobs=torch.tensor(logprobs, dtype=torch.float64, device="cuda"))
