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


@pytest.mark.gpu
def test_strides_of_one_element(dev):
    """A dimension of one element has no stride that matters: one new token, one key head, one page."""
    b = paged.Batch([5], [1], 2, 1, 64, 16, seed=1, spare_pages=0)
    want = ds.dflash_paged_attention(*b.args())
    q = b.query.as_strided(b.query.shape, (3, b.query.stride(1), 1), b.query.storage_offset())
    s = b.key_cache.stride()
    kc = b.key_cache.as_strided(b.key_cache.shape, (1, s[1], 7, 1))
    vc = b.value_cache.as_strided(b.value_cache.shape, (5, s[1], 64, 1))
    got = ds.dflash_paged_attention(q, kc, vc, *b.args()[3:])
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    x = torch.randn((1, 1, 64), device=dev).to(BF)
    slot = torch.tensor([9], device=dev)
    ds.dflash_store_kv(x.as_strided(x.shape, (3, 5, 1)), x.as_strided(x.shape, (1, 1, 1)), slot, kc, vc)
    assert torch.equal(b.key_cache[0, 9], x[0]) and torch.equal(b.value_cache[0, 9], x[0])
    assert ds.dflash_device_status(clear=True) == 0
