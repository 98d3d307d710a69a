"""Scores, weights and row statistics of the paged attention where they could be lost: far from
zero, far from one another, capped at any height. Against plain 64-bit forms (tests/paged.py)."""

from __future__ import annotations

import pytest
import torch

import paged
import draft_candidate_selector_gb300 as ds

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(BF, None), (FP, None), (BF, E4), (FP, E4)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    ds.dflash_device_status(clear=True)
    return d


def put(b: paged.Batch, r: int, keys=None, values=None):
    """Request r's keys or values [kv, Hkv, D] (as the cache is to hold them, before its scale), in
    the batch's plain lists and in its cache."""
    for x, rows, cache in ((keys, b.k, b.key_cache), (values, b.v, b.value_cache)):
        if x is None:
            continue
        rows[r] = x = x.to(b.cache_dtype)
        raw, y = (cache.view(torch.uint8), x.view(torch.uint8)) if b.small else (cache, x)
        for at in range(0, len(x), b.page):
            part = y[at:at + b.page].to(cache.device)
            raw[int(b.table[r, at // b.page]), :len(part)] = part


def set_queries(b: paged.Batch, x: torch.Tensor):
    b.qkv[:, :b.Hq] = x.to(b.dtype)
    b.query.copy_(b.qkv[:, :b.Hq])


def attend(b, left=-1, right=0, softcap=0.0, **kw):
    got = ds.dflash_paged_attention(*b.args(), window_left=left, window_right=right,
                                    softcap=softcap, **b.scales(), **kw)
    assert ds.dflash_device_status(clear=True) == 0
    return got


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("loud", [1.0, 2.0 ** 9])
def test_scores_far_below_zero(dev, dtype, cache, D, loud):
    """Prompts of one row tile and one key tile whose visible scores all lie below -100: the maximum
    is theirs, whatever else the halves of a CTA pass to one another. `loud` moves the size from
    the keys to the queries."""
    g = torch.Generator().manual_seed(D)
    new = [20] * 40 + [3, 32, 9]
    b = paged.Batch([0] * len(new), new, 4, 1, D, 16, dtype, cache, seed=1)
    u = torch.where(torch.rand(D, generator=g) < 0.5, -1.0, 1.0)
    # score = scale D a c with scale D = sqrt(D): between -100 and -200
    a = loud * (1 + torch.rand((b.T, b.Hq, 1), generator=g))
    set_queries(b, a * u)
    for r, n in enumerate(new):
        c = -100.0 / (D ** 0.5 * loud * b.k_scale) * (1 + 0.05 * torch.rand((n, 1, 1), generator=g))
        put(b, r, keys=c * u)
    want = paged.attention(b)
    assert want[1].max() < -90
    for _ in range(5):
        paged.assert_attention(attend(b), want)


def reference(b, left=-1, right=0, softcap=0.0, quick=0.0, step=0.0):
    """fp64 (out, lse) and bounds, with the unit roundoffs of paged.attention, but a score bound that
    is relative: a score's fp32 sum of D products is off by at most (D + 8) 2^-23 sum|q k| scale,
    which the cap (of slope 1 at most) does not enlarge; the cap itself adds 2^-19 of the capped
    score and `quick`, and rounding 2^-22 of it. `step`: half the smallest step of a weight, of the
    largest."""
    u = 2.0 ** -8 if b.dtype == BF else 2.0 ** -11
    g = b.Hq // b.Hkv
    out = torch.zeros((b.T, b.Hq, b.D), dtype=torch.float64)
    lse = torch.zeros((b.T, b.Hq), dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    for r in range(len(b.ctx)):
        n, L = int(b.new[r]), int(b.kv[r])
        kr, vr = b.k[r].double() * b.k_scale, b.v[r].double() * b.v_scale
        pos, j = torch.arange(L - n, L)[:, None], torch.arange(L)[None, :]
        see = torch.ones((n, L), dtype=torch.bool)
        if right >= 0:
            see &= j <= pos + right
        if left >= 0:
            see &= j >= pos - left
        for h in range(b.Hq):
            q, k, v = b.qkv[t0:t0 + n, h].double(), kr[:, h // g], vr[:, h // g]
            s = q @ k.T * b.D ** -0.5
            ds_ = (b.D + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) * b.D ** -0.5
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
                ds_ = ds_ + 2.0 ** -19 * s.abs() + quick
            ds_ = (ds_ + 2.0 ** -22 * s.abs()).masked_fill(~see, 0.0).amax(1, keepdim=True)
            s = s.masked_fill(~see, -torch.inf)
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m)
            tot = p.sum(1, keepdim=True)
            o, A = p @ v / tot, p @ v.abs() / tot
            sums = (L + 64) * 2.0 ** -22
            at = slice(t0, t0 + n)
            out[at, h], lse[at, h] = o, (m + torch.log(tot))[:, 0]
            tol[at, h] = (u * o.abs() + (u + 2 * ds_ + sums) * A
                          + step * (see.double() @ v.abs()) / tot + 1e-30)
            tol_lse[at, h] = ds_[:, 0] + sums + 2.0 ** -22 * lse[at, h].abs()
        t0 += n
    return out, lse, tol, tol_lse


@pytest.mark.parametrize("softcap", [0.5, 64.0, 65.0, 1e3, 1e4, 1e6, 1e30, 3.4e38])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D,few", [(64, True), (128, True), (64, False), (128, False), (80, True)])
def test_caps_of_any_height(dev, softcap, dtype, cache, D, few):
    """A cap costs a score no more than its own rounding, or 2^-21 of a cap up to 64: single keys,
    whose log-sum-exp is the score, and more."""
    new = [1] * 50 + [2, 1] if few else [40, 17, 33]
    ctx = [0] * 50 + [3, 300] if few else [0, 5, 290]
    b = paged.Batch(ctx, new, 4, 2, D, 16, dtype, cache, seed=D, spread=3.0)
    # fp16 weights have 2^-24 as their smallest step, and are taken of a maximum that is at most 1
    step = 0.0 if dtype == BF and cache is None else 2.0 ** -25
    want = reference(b, softcap=softcap, quick=2.0 ** -21 * softcap if softcap <= 64 else 0.0, step=step)
    paged.assert_attention(attend(b, softcap=softcap), want)


@pytest.mark.parametrize("dtype,cache", TYPES[1:])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40])
def test_small_weights_keep_their_mass(dev, dtype, cache, D, n):
    """One key 18 nats above 20000 others, which hold all of the output: weights of 2^-26 in fp16."""
    b = paged.Batch([20000], [n], 4, 1, D, 64, dtype, cache, seed=2)
    L = 20000 + n
    q = torch.zeros((n, 4, D))
    q[:, :, 0] = D ** 0.5
    keys, values = torch.zeros((L, 1, D)), torch.ones((L, 1, D))
    keys[5, 0, 0] = 18.0
    values[5] = 0.0
    set_queries(b, q)
    put(b, 0, keys / b.k_scale, values / b.v_scale)
    # Equal requests over the same pages, in whole items of one SM each: parts of a long item have
    # maxima of their own, and only the first would meet the small weights.
    R = 304 if n == 1 else 152
    args = (b.query.repeat(R, 1, 1), b.key_cache, b.value_cache, b.block_table.repeat(R, 1),
            torch.arange(R + 1, dtype=torch.int32, device=dev) * n, b.kv_lens.repeat(R))
    out, lse = ds.dflash_paged_attention(*args, **b.scales())
    # Of the largest weight at the least: 2^-39 where it is 2^14 (few rows), 2^-32 where it is 2^7.
    want = reference(b, step=2.0 ** -39 if n == 1 else 2.0 ** -32)
    assert want[0].max() < 1e-3
    for r in range(0, R, 19):
        paged.assert_attention((out[r * n:(r + 1) * n], lse[r * n:(r + 1) * n]), want, f"copy {r}")
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128, 80])
@pytest.mark.parametrize("ctx,new", [(600, 3), (600, 40), (20000, 3), (5000, 300)])
def test_bad_pages_reach_only_rows_that_see_them(dev, dtype, cache, D, ctx, new):
    """Pages that a window has left may be taken back (id -1): nothing is recorded and nothing
    changes. A bad page that some rows see makes NaN of those rows alone."""
    left = 50
    b = paged.Batch([ctx, 70], [new, 9], 4, 2, D, 16, dtype, cache, seed=3)
    kw = dict(window_left=left, window_right=0, **b.scales())
    want = ds.dflash_paged_attention(*b.args(), **kw)
    assert ds.dflash_device_status(clear=True) == 0
    table = b.block_table.clone()
    hidden = (ctx - left) // 16                      # pages of which no row sees a key
    b.block_table[0, :hidden] = torch.tensor([-1, 2 ** 31 - 1], dtype=torch.int32,
                                             device=dev).repeat(hidden)[:hidden]
    for g, w in zip(ds.dflash_paged_attention(*b.args(), **kw), want):
        assert torch.equal(g, w)
    assert ds.dflash_device_status(clear=True) == 0
    for page in sorted({hidden, hidden + 1, ctx // 16, (ctx + new - 1) // 16}):
        b.block_table.copy_(table)
        b.block_table[0, page] = -1
        got = ds.dflash_paged_attention(*b.args(), **kw)
        assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_ID
        pos = torch.arange(ctx, ctx + new, device=dev)
        sees = torch.cat([(pos - left < 16 * page + 16) & (pos >= 16 * page),
                          torch.zeros(9, dtype=torch.bool, device=dev)])
        assert sees.any()
        for g, w in zip(got, want):
            assert torch.isnan(g[sees]).all()
            assert torch.equal(g[~sees], w[~sees])
