"""Plain 64-bit forms of the paged key-value cache operators, and inputs for their tests.

Nothing here uses the library. The tables are Python loops over requests and tokens, the
attention a loop over requests and heads in fp64 that gathers only the keys a row may see.
"""

from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- block tables

def tables(ctx, new, held, free, table, page, T):
    """(table, query_start, kv_lens, held_out, positions, slots, needed, refused) of one step."""
    table = table.copy()
    R, width = table.shape
    start, kv, held_out, refused = [0], [], [], []
    positions, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    taken = 0
    for r in range(R):
        c, n, h = int(ctx[r]), int(new[r]), int(held[r])
        fits = (c >= 0 and n >= 0 and 0 <= h <= width and c <= h * page
                and -(-(c + n) // page) <= width)
        need = max(0, -(-(c + n) // page) - h) if fits else 0
        granted = fits and (need == 0 or taken + need <= len(free))
        if granted and need:
            table[r, h:h + need] = free[taken:taken + need]
        taken += need
        for i in range(min(max(n, 0), max(0, T - start[-1]))):
            t = start[-1] + i
            positions[t] = c + i
            if granted:
                slots[t] = int(table[r, (c + i) // page]) * page + (c + i) % page
        start.append(start[-1] + max(n, 0))
        kv.append(c + n if granted else 0)
        held_out.append(h + need if granted else h)
        refused.append(not granted)
    start = np.minimum(start, 2 ** 31 - 1)
    return (table, start, np.array(kv), np.array(held_out), positions, slots, taken,
            np.array(refused))


# ---------------------------------------------------------------- attention

class Batch:
    """A ragged batch over a paged cache on one device, every page of the pool in a random place.

    ctx, new: cached and new tokens of each request. Pool rows that no request uses, and rows
    behind a request's last token, hold `junk`.
    """

    def __init__(self, ctx, new, Hq, Hkv, D, page, dtype=torch.bfloat16, cache=None,
                 layout="nhd", seed=0, device="cuda", junk=float("nan"), spread=1.0,
                 spare_pages=3, first_page=0):
        self.ctx, self.new = np.asarray(ctx), np.asarray(new)
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.cache_dtype = cache or dtype
        self.small = self.cache_dtype == E4M3
        self.k_scale, self.v_scale = (0.25, 0.125) if self.small else (1.0, 1.0)
        g = torch.Generator().manual_seed(seed)
        R = len(self.ctx)
        self.kv = self.ctx + self.new
        need = -(-self.kv // page)
        pool = int(need.sum()) + spare_pages + first_page
        self.max_pages = max(1, int(need.max()))
        order = torch.randperm(pool - first_page, generator=g) + first_page
        table = torch.full((R, self.max_pages), 0, dtype=torch.int32)
        at = 0
        for r in range(R):
            table[r, :need[r]] = order[at:at + need[r]].to(torch.int32)
            at += int(need[r])
        self.table = table
        T = int(self.new.sum())
        self.T = T
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g)
        qkv[:, :Hq] *= spread
        self.qkv = qkv.to(dtype)
        shape = (pool, Hkv, page, D) if layout == "hnd" else (pool, page, Hkv, D)
        self.k, self.v = [], []       # per request, [kv, Hkv, D] as held
        caches = []
        for rows in (self.k, self.v):
            c = torch.full(shape, 1.0).to(self.cache_dtype)
            if self.small:
                c.view(torch.uint8).fill_(0x7f if math.isnan(junk) else 0x7e)
            else:
                c.fill_(junk)
            cc = c.transpose(1, 2) if layout == "hnd" else c
            raw = cc.view(torch.uint8) if self.small else cc
            for r in range(R):
                x = torch.randn((int(self.kv[r]), Hkv, D), generator=g)
                x = (x / 0.2).clamp(-448, 448).to(E4M3) if self.small else x.to(dtype)
                rows.append(x)
                y = x.view(torch.uint8) if self.small else x
                for b in range(int(need[r])):
                    part = y[b * page:(b + 1) * page]
                    raw[int(table[r, b]), :part.shape[0]] = part
            caches.append(c)
        self.key_cache, self.value_cache = (c.to(device) for c in caches)
        if layout == "hnd":
            self.key_cache = self.key_cache.transpose(1, 2)
            self.value_cache = self.value_cache.transpose(1, 2)
        self.query = self.qkv.to(device)[:, :Hq]
        self.block_table = table.to(device)
        self.query_start = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]),
                                        dtype=torch.int32, device=device)
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device=device)

    def args(self):
        return (self.query, self.key_cache, self.value_cache, self.block_table, self.query_start,
                self.kv_lens)

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)


def attention(b: Batch, scale=None, left=-1, right=0, softcap=0.0):
    """fp64 (out, lse) and bounds on what a kernel may be off them.

    The kernel sums fp32 products and rounds the weights and the output to the query's type, of
    unit roundoff u: half the spacing 2^-7 of bf16's 8 significant bits, 2^-8, and
    2^-11 for fp16's 11. With A = sum_j p_j |v_j| / sum_j p_j:
      * a score's fp32 sum of D products is off by at most ds = (D + 8) 2^-23 sum|q k| scale,
        plus 2^-20 softcap for the cap's own functions, plus 2^-22 |s| for the rounding of the
        score itself and of its product with log2(e); a weight is then off by ds (relative),
        and the quotient by 2 ds A;
      * a rounded weight is off by u (relative), or 2^-25 of the largest where fp16 has no
        smaller step, so the output by u A + 2^-25 sum|v| / sum p;
      * fp32 exponentials and sums add (L + 64) 2^-22 A; the output's rounding adds u |out|.
    lse: the largest ds, the sums' (L + 64) 2^-22, and its own rounding.
    """
    scale = b.D ** -0.5 if scale is None else scale
    u = 2.0 ** -8 if b.dtype == torch.bfloat16 else 2.0 ** -11
    g = b.Hq // b.Hkv
    out = torch.zeros((b.T, b.Hq, b.D), dtype=torch.float64)
    lse = torch.full((b.T, b.Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.full_like(out, 1e-30), torch.full_like(lse, 1e-30)
    t0 = 0
    for r in range(len(b.ctx)):
        n, L = int(b.new[r]), int(b.kv[r])
        if L and n:
            kr, vr = b.k[r].double() * b.k_scale, b.v[r].double() * b.v_scale
            pos = torch.arange(L - n, L)[:, None]
            j = torch.arange(L)[None, :]
            see = torch.ones((n, L), dtype=torch.bool)
            if right >= 0:
                see &= j <= pos + right
            if left >= 0:
                see &= j >= pos - left
            for h in range(b.Hq):
                q, k, v = b.qkv[t0:t0 + n, h].double(), kr[:, h // g], vr[:, h // g]
                raw = q @ k.T * scale
                ds = (b.D + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) * scale
                s = softcap * torch.tanh(raw / softcap) if softcap > 0 else raw
                ds = ds + 2.0 ** -20 * softcap + 2.0 ** -22 * s.abs()
                s = s.masked_fill(~see, -math.inf)
                ds = ds.masked_fill(~see, 0.0).amax(1, keepdim=True)
                m = s.amax(1, keepdim=True)
                m = torch.where(m == -math.inf, torch.zeros_like(m), m)
                p = torch.exp(s - m)
                tot = p.sum(1, keepdim=True)
                safe = torch.where(tot == 0, torch.ones_like(tot), tot)
                vz = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))
                o = p @ vz / safe
                A = p @ vz.abs() / safe
                seen_v = see.double() @ vz.abs()
                out[t0:t0 + n, h] = o
                lse[t0:t0 + n, h] = (m + torch.log(tot))[:, 0]
                small = 2.0 ** -25 * seen_v / safe if u < 2.0 ** -10 else 0.0
                tol[t0:t0 + n, h] = (u * o.abs() + (u + 2 * ds + (L + 64) * 2.0 ** -22) * A
                                     + small + 1e-30)
                tol_lse[t0:t0 + n, h] = (ds[:, 0] + (L + 64) * 2.0 ** -22
                                         + 2.0 ** -22 * lse[t0:t0 + n, h].abs().nan_to_num(0, 0, 0))
        t0 += n
    return out, lse, tol, tol_lse


def assert_attention(got, want, what=""):
    out, lse = (t.double().cpu() for t in got)
    o, z, tol, tol_z = want
    assert torch.isfinite(out).all(), f"{what}: {int((~torch.isfinite(out)).sum())} non-finite"
    far = (out - o).abs() / tol
    assert far.max() <= 1, f"{what}: out off by {float(far.max()):.3g} of its bound"
    assert torch.equal(torch.isinf(lse), torch.isinf(z)), f"{what}: empty rows differ"
    keep = ~torch.isinf(z)
    if keep.any():
        far = (lse[keep] - z[keep]).abs() / tol_z[keep]
        assert far.max() <= 1, f"{what}: lse off by {float(far.max()):.3g} of its bound"
