"""Calls of the paged operators as users make them: workspaces, caller-given outputs, layouts with
dimensions of one element, tensors of several devices."""

from __future__ import annotations

import pytest
import torch

import paged
import draft_candidate_selector_gb300 as ds

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    ds.dflash_device_status(clear=True)
    return d


@pytest.mark.gpu
def test_no_workspace_where_none_is_used(dev):
    """Head sizes of the CUDA-core kernel, which writes its outputs at once."""
    for D in (8, 80, 96, 192, 256):
        assert 0 < ds.dflash_paged_attention_workspace_bytes(3, 9, 8, 2, D) <= 256
    assert 0 < ds.dflash_paged_attention_workspace_bytes(3, 9, 130, 1, 128) <= 256
    b = paged.Batch([30, 3000], [5, 1], 4, 2, 256, 16, seed=2)
    got = ds.dflash_paged_attention(*b.args(), workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    paged.assert_attention(got, paged.attention(b))
    assert ds.dflash_device_status(clear=True) == 0
