"""The example's loop: prompts and drafted blocks through the paged cache and the selector."""

from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

import draft_candidate_selector_gb300 as ds

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "draft_loop.py")


@pytest.fixture(scope="module")
def loop():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("draft_loop", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    ds.dflash_device_status(clear=True)
    return module


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_page_size_does_not_matter(loop, cache):
    """Key tiles are 128 tokens for every page size, so the drafts agree bit for bit."""
    want = loop.run(5, 300, 3, 16, cache)
    for page in (32, 128):
        got = loop.run(5, 300, 3, page, cache)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(want[1]).all()
    assert ds.dflash_device_status(clear=True) == 0


def test_hidden_states_match_dense_attention(loop):
    """One block behind cached prompts, against fp64 attention over the same bf16 rows."""
    R, S, lens = 3, 15, [1, 130, 257]
    d = loop.Drafter(R, 100, 16, 400, window=100)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(4096, (n,), generator=g).cuda() for n in lens]
    d.prompts(prompts)
    assert d.context.tolist() == lens
    block = torch.randint(4096, (R, 1 + S), generator=g).cuda()
    new = torch.full((R,), 1 + S, dtype=torch.int32, device="cuda")
    got = d.attend(block.view(-1), new, window_right=-1).view(R, 1 + S, -1)
    hq, hkv, D = d.heads
    for r in range(R):
        tokens = torch.cat([prompts[r], block[r]])
        x = d.embedded(tokens, torch.arange(len(tokens), device="cuda"))
        # Rows of this product may differ by a bf16 rounding from the batch's, where the
        # library sums in another order.
        q, k, v = (x @ d.w_qkv.t()).view(len(x), hq + 2 * hkv, D).double().split([hq, hkv, hkv], 1)
        k, v = k.repeat_interleave(hq // hkv, 1), v.repeat_interleave(hq // hkv, 1)
        n, L = 1 + S, len(x)
        s = torch.einsum("ihd,jhd->hij", q[-n:], k) / math.sqrt(D)
        s = d.softcap * torch.tanh(s / d.softcap)
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        s = s.masked_fill(torch.arange(L, device="cuda")[None] < pos - 99, -math.inf)
        attn = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, -1)
        want = x[-n:].double() + attn @ d.w_out.double().t()
        # bf16 rounds queries, keys, values, the weights, the attention, its product and the sum,
        # each by 2^-8 of values that are sums of unit variance: a few 2^-8 of the largest.
        assert (got[r].double() - want).abs().max() <= 16 * 2.0 ** -8 * want.abs().max()
    assert ds.dflash_device_status(clear=True) == 0


def test_out_of_pages(loop):
    d = loop.Drafter(2, 3, 16, 400)
    with pytest.raises(RuntimeError, match="out of pages"):
        d.prompts([torch.zeros(40, dtype=torch.long, device="cuda")] * 2)
    ds.dflash_device_status(clear=True)


def test_earlier_faults_are_not_passed_over(loop):
    """A device status set in front of a step's tables (here by a store to a slot outside the cache)
    is an error of the loop, not cleared and forgotten."""
    d = loop.Drafter(2, 30, 16, 400)
    x = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    ds.dflash_store_kv(x, x, torch.tensor([30 * 16], device="cuda"), d.k_cache, d.v_cache)
    with pytest.raises(RuntimeError, match="status"):
        d.prompts([torch.zeros(40, dtype=torch.long, device="cuda")] * 2)
    assert ds.dflash_device_status(clear=True) == 0
