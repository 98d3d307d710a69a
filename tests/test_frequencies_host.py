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


@pytest.mark.parametrize("kw", [dict(base=5e-324), dict(base=5e-324, factor=2.0, original_len=4096.0),
                                dict(factor=1e-310), dict(base=1e-300, factor=1e-300, original_len=64.0),
                                dict(base=1e-300, factor=1e-20)])
def test_frequencies_that_are_no_numbers(kw):
    """A base or a factor so small that a frequency is infinite is refused, with the pair's number."""
    with pytest.raises(ValueError, match=r"pair \d+"):
        ds.dflash_rope_frequencies(128, device="cpu", **kw)
    out = ds.dflash_rope_frequencies(128, base=1e-4, factor=1e-3, device="cpu")
    near(out.tolist(), [(1e-4 ** (-2 * j / 128)) / 1e-3 for j in range(64)])
