"""Tokens without any probability are never drawn, however near the number is to a border."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import draft_candidate_selector_gb300 as ds
from test_sampling_gpu import BF, F32, FP, INF, Batch, clean, dev   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [0, 1500, 6000, -9])
@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_tiles_that_the_draft_takes_whole(dev, dtype, at):                            # noqa: F811
    """All tokens of a tile that are not masked are the draft's, and likelier under it: nothing of the tile is
    left, though a rounding of its sum may be. The number is 0, or the last below 1."""
    R, V, K = 200, 20008, 8                              # rows of whole vectors: tiles from 0 on
    b = Batch(dev, [2] * R, V, 1, K, dtype, spread=1.5, likely=False, seed=3)
    g = torch.Generator(device=dev).manual_seed(at + 50)
    tile = 4096 // b.logits.element_size()
    first = (V + at if at < 0 else at) // tile * tile
    x = b.logits.float()
    inside = torch.arange(V, device=dev) // tile == first // tile
    x[:, inside] = -INF
    n = int(inside.sum())
    ids = first + torch.rand((R, n), generator=g, device=dev).argsort(1)[:, :K]
    x[::2].scatter_(1, ids, 9 + 1.5 * torch.randn((R, K), generator=g, device=dev))
    x[:, ::3] = torch.where(inside[::3], x[:, ::3], torch.full_like(x[:, ::3], -INF))
    b.logits = x.to(dtype)
    p = torch.softmax(b.logits[::2].double(), 1).gather(1, ids)
    b.ids, b.probs = ids.to(torch.int32)[:, None].contiguous(), (p / p.sum(1, keepdim=True)).float()[:, None].contiguous()
    b.drafts = b.ids[:, :, 0].contiguous()
    b.accept.fill_(1 - 2.0 ** -24)
    assert (b.probs[:, 0].double() > p).all()
    for u in (0.0, 1 - 2.0 ** -24):
        b.sample.fill_(u)
        got = b.check()
        assert (got[1] == 1).all()
        x = b.logits[::2].gather(1, got[0][:, :1].long())
        assert torch.isfinite(x).all() and not (got[0][:, :1] == b.ids[:, 0]).any()


@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_little_left_beside_a_tile(dev, dtype, where):                                # noqa: F811
    """All but about 2^-30 of a row is in one tile, which the draft takes whole; rounding is 2^-46 of the row, far more
    than from the border to the end of what is left. That is four like tokens in a tile far behind or before."""
    R, V, K = 200, 20008, 8
    b = Batch(dev, [2] * R, V, 1, K, dtype, likely=False, seed=5)
    g = torch.Generator(device=dev).manual_seed(9)
    tile = 4096 // b.logits.element_size()
    first, other = (0, 15000) if where == "first" else (V // tile * tile, 2100)
    ids = first + torch.rand((R, min(tile, V - first)), generator=g, device=dev).argsort(1)[:, :K]
    x = torch.full((2 * R, V), -INF, device=dev)
    top = 8 + 1.5 * torch.randn((R, K), generator=g, device=dev)
    x[::2].scatter_(1, ids, top)
    x[::2, other:other + 40:10] = (top.logsumexp(1) - 22.2)[:, None]
    x[1::2, 7] = 0.0
    b.logits = x.to(dtype)
    p = torch.softmax(b.logits[::2].double(), 1).gather(1, ids)
    b.ids, b.probs = ids.to(torch.int32)[:, None].contiguous(), (p * 1.0001).float()[:, None].contiguous()
    b.drafts = b.ids[:, :, 0].contiguous()
    b.accept.fill_(1 - 2.0 ** -24)
    for u, token in ((0.0, other), (1 - 2.0 ** -24, other + 30)):
        b.sample.fill_(u)
        assert (b.check()[0][:, 0] == token).all()


@pytest.mark.parametrize("K", [7, 13, 32])
def test_masked_candidates(dev, K):                                                   # noqa: F811
    """A path's rows of equal parts with masked candidates between them, numbers that are borders between the
    parts: sums in another order differ in their last bit, which must not let a masked candidate in."""
    R = 4000
    g = torch.Generator(device=dev).manual_seed(K)
    n = (K - 1) // 2
    part = torch.randn((R, n), generator=g, device=dev)
    row = torch.full((R, K), -INF, device=dev)
    row[:, :n], row[:, n + 1:2 * n + 1] = part, part
    edges = row[:, None, None, :].expand(R, 1, K, K).contiguous()
    ids = torch.arange(K, dtype=torch.int32, device=dev).expand(R, 1, K).contiguous()
    path, _, probs = ds.dflash_sample_path(edges, ids, torch.full((R, 1), 0.5, device=dev))
    of_pick = probs[:, 0].gather(1, path.long())
    assert (of_pick > 0).all(), int((of_pick == 0).sum())
    # exact sums: the first of the second part; off by a rounding, the last of the first part
    assert ((path == n + 1) | (path == n - 1)).all()
    clean()
