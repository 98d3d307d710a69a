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
