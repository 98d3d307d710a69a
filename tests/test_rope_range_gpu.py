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
