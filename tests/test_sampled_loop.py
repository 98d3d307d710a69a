"""The example's loop with drawn drafts and a target model that verifies them: norm, rotation and store,
attention, selector, drawn paths and verification together."""

from __future__ import annotations

import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import step
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
@pytest.mark.parametrize("temperature", [0.0, 0.9])
def test_page_size_does_not_matter(loop, cache, temperature):
    """Runs of one seed agree bit for bit, over pages of any size."""
    want = loop.run_sampled(5, 200, 3, 16, cache, temperature=temperature)
    for page in (16, 64):
        got = loop.run_sampled(5, 200, 3, page, cache, temperature=temperature)
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    for tokens, counts, logprobs in want:
        at = torch.arange(16, device=tokens.device)
        assert ((tokens >= 0) == (at < counts[:, None])).all() and (counts >= 1).all()
        assert (logprobs <= 0).all() and ((logprobs == 0) | (at < counts[:, None])).all()


def test_a_step_against_the_plain_forms(loop):
    """One step's path and verification against the 64-bit forms on the same scores and logits, and its hidden
    states against dense fp64 attention over normed and rotated heads."""
    R, S, lens = 3, 15, [2, 90, 161]
    d = loop.Drafter(R, 100, 16, 400, seed=3, rotary=True, window=400, softcap=0.0)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(4096, (n,), generator=g).cuda() for n in lens]
    d.prompts(prompts)
    last = torch.randint(4096, (R,), generator=g).cuda()
    u = [torch.rand(s, generator=g).cuda() for s in ((R, S), (R, S), (R,))]
    ids, edges = d.candidates(last)
    path, drafts, probs = ds.dflash_sample_path(edges, ids, u[0], temperature=0.7)
    want, _ = step.sample_path(edges, u[0], [0.7] * R)
    np.testing.assert_array_equal(path.cpu().numpy(), want)
    logits, start = d.logits(last, drafts)
    tokens, counts, _ = ds.dflash_verify_drafts(logits, start, drafts, u[1], u[2], ids, probs, temperature=0.9)
    want = step.verify(logits, start, drafts, u[1], u[2], ids, probs, [0.9] * R)
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
    np.testing.assert_array_equal(counts.cpu().numpy(), want[1])

    hq, hkv, D = d.heads
    new = torch.full((R,), 1 + S, dtype=torch.int32, device="cuda")
    block = torch.cat([last[:, None], drafts.long()], 1)
    got = d.attend(block.view(-1), new, window_right=0).view(R, 1 + S, -1)
    f = d.frequencies.tolist()
    for r in range(R):
        x = d.embed[torch.cat([prompts[r], block[r]])]
        q, k, v = (x @ d.w_qkv.t()).view(len(x), hq + 2 * hkv, D).split([hq, hkv, hkv], 1)
        turns = step.turns(range(len(x)), f)
        q, _ = step.norm_rope(q, d.q_weight, 1e-6, turns, False, 1.0)
        k, _ = step.norm_rope(k, d.k_weight, 1e-6, turns, False, 1.0)
        k, v = k.repeat_interleave(hq // hkv, 1), v.cpu().double().repeat_interleave(hq // hkv, 1)
        n, L = 1 + S, len(x)
        s = torch.einsum("ihd,jhd->hij", q[-n:], k) / math.sqrt(D)
        s = s.masked_fill(torch.arange(L)[None] > torch.arange(L - n, L)[:, None], -math.inf)
        attn = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, -1)
        want = x[-n:].cpu().double() + attn @ d.w_out.cpu().double().t()
        # bf16 rounds queries, keys, values, the weights, the attention, its product and the sum,
        # each by 2^-8 of values that are sums of unit variance: a few 2^-8 of the largest.
        assert (got[r].cpu().double() - want).abs().max() <= 16 * 2.0 ** -8 * want.abs().max()
    assert ds.dflash_device_status(clear=True) == 0
