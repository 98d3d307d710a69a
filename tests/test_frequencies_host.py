"""Rotation frequencies at the ends of their range, on the host."""

from __future__ import annotations

import pytest
import torch

import draft_candidate_selector_gb300 as ds
from test_step_host import near


def test_backward_turns():
    """A negative frequency is its positive one's, negated, and as near to what was given."""
    f = torch.tensor([1e-6, 1e-9, 3e-12, 0.3, 1.0, 6.5, 100.0, 12345.678], dtype=torch.float64)
    forward = ds.dflash_rope_frequencies(16, inv_freq=f, device="cpu")
    backward = ds.dflash_rope_frequencies(16, inv_freq=-f, device="cpu")
    assert torch.equal(backward, -forward)
    near(forward.tolist(), f.tolist())
    near(backward.tolist(), (-f).tolist())
