"""The norm over the whole range of its inputs, and values that are not rotated."""

from __future__ import annotations

import pytest
import torch

import step
import draft_candidate_selector_gb300 as ds
from test_rope_gpu import BF, FP, Case, caches, clean, dev   # noqa: F401

pytestmark = pytest.mark.gpu


def fp32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def spread(c, powers, seed=0):
    """Token t's heads get an rms of about 2^powers[t]: tokens of all magnitudes lie side by side."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(c.qkv.shape, generator=g, dtype=torch.float64)
    top = torch.finfo(c.dtype).max
    for t, p in enumerate(powers):
        x[t] *= 2.0 ** p
    c.qkv.copy_(x.clamp(-top, top).to(c.dtype))


def check_norm(c, eps):
    for x, w, y in zip((c.query, c.key), (c.q_weight, c.k_weight), c.run(eps=eps)):
        step.close_heads(y, *c.want(x, w, fp32(eps)), c.dtype)
    clean()


@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("eps", [1e-6, 1e-5, 1e-3, 0.0, 1e30])
def test_squares_past_the_range(dev, D, eps):                                         # noqa: F811
    """Heads whose sum of squares passes fp32's range, whose eps is as small beside it as the formula says."""
    powers = [60, 0, 60.5, 61, 1, 61.5, 62, 63, -2, 64, 66, 68, 3, 70, 74, 90, 126, 59, 58]
    c = Case(dev, len(powers), 3, 2, D)
    spread(c, powers, D)
    check_norm(c, eps)
    for t in (0, 3, 9):                              # equal values
        c.qkv[t] = 2.0 ** powers[t]
    check_norm(c, eps)


def test_squares_past_the_range_with_the_store(dev):                                  # noqa: F811
    powers = [60, 0, 61, 62, -1, 64, 68, 74]
    c = Case(dev, len(powers), 3, 2, 128)
    spread(c, powers)
    kc, vc = caches(dev, 3, 16, 2, 128, BF)
    q, _, _ = ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc, eps=1e-6, **c.how)
    step.close_heads(q, *c.want(c.query, c.q_weight, fp32(1e-6)), BF)
    step.close_heads(kc.flatten(0, 1)[c.slots], *c.want(c.key, c.k_weight, fp32(1e-6)), BF)
    clean()


@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-20, 1e-6])
def test_squares_below_the_range(dev, D, eps):                                        # noqa: F811
    """Heads whose squares are below fp32's range, with an eps that is as small; with none, a head of zeros has no
    norm, as the formula says."""
    powers = [-49, 0, -50, -52, -60, 3, -63, -70, -72, -74, 61, -75, -80, -100, -110, -1, -126, 126]
    c = Case(dev, len(powers), 3, 2, D)
    spread(c, powers, D)
    check_norm(c, eps)
    c.qkv[4] = 0
    got = c.run(eps=eps)[0]
    assert torch.isnan(got[4]).all() if eps == 0 else not got[4].any()
    assert torch.isfinite(got[torch.arange(len(powers)) != 4]).all()
    clean()


def test_small_fp16_values(dev):                                                      # noqa: F811
    c = Case(dev, 6, 3, 2, 128, FP)
    spread(c, [-24, -20, -14, 0, 8, 14])
    c.qkv[c.qkv == 0] = 2.0 ** -24
    check_norm(c, 0.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(128, 64), (128, 2), (64, 62), (248, 34), (80, 20), (96, 0), (256, 16)])
def test_values_behind_the_rotated_ones(dev, D, rotary, interleaved):                 # noqa: F811
    """Without a norm they stay as they are: infinities, NaN and -0 among them, none of which reaches another."""
    for dtype in (BF, FP):
        c = Case(dev, 5, 3, 2, D, dtype, rotary, interleaved, norm="")
        want = [x.clone() for x in c.run()]
        g = torch.Generator().manual_seed(D)
        odd = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 0.0])
        which = torch.randint(0, 10, (5, 7, D - rotary), generator=g)
        tail = c.qkv[:, :, rotary:].cpu()
        tail = torch.where(which < 5, odd[which.clamp(max=4)].to(dtype), tail)
        c.qkv[:, :, rotary:] = tail.to(dev)
        kc, vc = caches(dev, 2, 16, 2, D, dtype)
        stored = ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc, **c.how)
        for got in (c.run(), (stored[0], kc.flatten(0, 1)[c.slots])):
            for x, y, w in zip((c.query, c.key), got, want):
                assert torch.equal(y[..., :rotary], w[..., :rotary])
                x, y = x[..., rotary:].contiguous(), y[..., rotary:].contiguous()
                assert torch.equal(torch.isnan(x), torch.isnan(y))
                bits = lambda v: v.nan_to_num(nan=1.0, posinf=2.0, neginf=3.0).view(torch.int16)     # noqa: E731
                assert torch.equal(torch.isinf(x), torch.isinf(y)) and torch.equal(bits(x), bits(y))
        clean()
