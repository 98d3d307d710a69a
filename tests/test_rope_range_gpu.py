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
