"""A block drafter's loop over a paged key-value cache: prompts enter, then blocks are drafted.

One attention layer of random weights stands for the drafter. Each step runs, on the current stream:

    dflash_block_tables      pages, positions and cache slots of the step's new tokens
    dflash_store_kv          their keys and values into the cache
    dflash_paged_attention   their attention over everything cached, themselves included
    dflash_selector_lmhead   candidates from the LM head, hidden projection, edge scores
    dflash_best_path         one drafted token per mask position

A block is a request's last token and S mask tokens, which see one another and a window of the
context (window_right -1). A step drafts S tokens; a verifier that takes a random number of them
stands for the target model. The tokens taken are the context of the next step, so the block's own
keys and values are written over.

    python examples/draft_loop.py --requests 8 --prompt 400 --steps 4
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_candidate_selector_gb300 as ds   # noqa: E402


def check_status() -> None:
    """Raises if a kernel of the calls so far has set a bit of the device status."""
    status = ds.dflash_device_status()
    if status & ds.DEVICE_NO_PAGES:
        raise RuntimeError("the cache is out of pages")
    if status:
        raise RuntimeError(f"device status {status:#x}")


class Drafter:
    """Weights, the paged cache and the requests' state. All tensors live on `device`."""

    def __init__(self, requests: int, pages: int, page_size: int, max_tokens: int, *,
                 q_heads=16, kv_heads=4, head_dim=64, vocab=4096, rank=64, K=8, S=15, window=1024,
                 softcap=50.0, cache_dtype=torch.bfloat16, seed=0, device="cuda"):
        self.R, self.page_size, self.S, self.K = requests, page_size, S, K
        self.heads, self.window, self.softcap = (q_heads, kv_heads, head_dim), window, softcap
        hidden = q_heads * head_dim
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(device, torch.bfloat16)

        self.embed = weight(vocab + 1, hidden) * hidden ** 0.5          # the last row: the mask token
        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = weight(hidden, hidden)
        self.lm_head = weight(vocab, hidden)
        self.w_proj = weight(rank, hidden)
        self.pred_cb, self.succ_cb = weight(vocab, rank), weight(vocab, rank)
        self.mask_token = vocab

        # The cache: one pool of pages for keys and one for values, and each request's page list.
        self.k_cache = torch.zeros(pages, page_size, kv_heads, head_dim, device=device).to(cache_dtype)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.k_scale, self.v_scale = ((0.05, 0.05) if cache_dtype == torch.float8_e4m3fn
                                      else (1.0, 1.0))
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.zeros(requests, -(-max_tokens // page_size), **i32)
        self.held = torch.zeros(requests, **i32)
        self.context = torch.zeros(requests, **i32)
        self.free = torch.arange(pages, **i32).flip(0).contiguous()

    def embedded(self, tokens: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        """Embeddings of tokens at positions, which sines tell apart."""
        n = self.embed.shape[1]
        wave = 0.1 ** (4 * torch.arange(n, device=positions.device) / n)
        return self.embed[tokens] + torch.sin(positions[:, None] * wave).to(torch.bfloat16)

    def attend(self, tokens: torch.Tensor, new_lens: torch.Tensor, window_right: int) -> torch.Tensor:
        """Hidden states [T, hidden] of new tokens [T], new_lens [R] of them for each request, behind
        the context of each; their keys and values are cached, the context is not moved on."""
        start, kv_lens, self.held, positions, slots, taken = ds.dflash_block_tables(
            self.context, new_lens, self.held, self.free, self.table, self.page_size, len(tokens))
        # The host reads two values a step: the number of pages taken, and the status word, which
        # holds what the kernels have met since it was last read (here, or after the last step).
        self.free = self.free[int(taken):].contiguous()
        check_status()
        hq, hkv, d = self.heads
        x = self.embedded(tokens, positions)
        q, k, v = (x @ self.w_qkv.t()).view(len(tokens), hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
        ds.dflash_store_kv(k, v, slots, self.k_cache, self.v_cache, self.k_scale, self.v_scale)
        out, _ = ds.dflash_paged_attention(
            q, self.k_cache, self.v_cache, self.table, start, kv_lens, window_left=self.window - 1,
            window_right=window_right, softcap=self.softcap, k_scale=self.k_scale,
            v_scale=self.v_scale)
        return x + out.view(len(tokens), -1) @ self.w_out.t()

    def prompts(self, prompts: list[torch.Tensor]) -> None:
        """Caches the requests' prompts, causally, and moves the contexts on."""
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=self.context.device)
        self.attend(torch.cat(prompts), lens, window_right=0)
        self.context = self.context + lens

    def draft(self, last: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
        """Tokens [R, S] drafted behind the requests' last tokens [R], and their paths' scores."""
        block = torch.full((self.R, 1 + self.S), self.mask_token, device=last.device)
        block[:, 0] = last
        new = torch.full((self.R,), 1 + self.S, dtype=torch.int32, device=last.device)
        x = self.attend(block.view(-1), new, window_right=-1)
        masks = x.view(self.R, 1 + self.S, -1)[:, 1:].contiguous()
        ids, _, _, edges = ds.dflash_selector_lmhead(masks, self.lm_head, self.w_proj, self.pred_cb,
                                                     self.succ_cb, last.to(torch.int32), self.K)
        _, tokens, score = ds.dflash_best_path(edges, ids)
        return tokens, score

    def take(self, count: torch.Tensor) -> None:
        """Moves the contexts on by the tokens taken (the last one and those that follow it)."""
        self.context = self.context + count.to(torch.int32)


def run(requests=8, prompt=400, steps=4, page_size=16, cache_dtype=torch.bfloat16, seed=0,
        device="cuda", show=False) -> tuple[torch.Tensor, torch.Tensor]:
    """Drafted tokens [steps, R, S] and scores [steps, R] of seeded prompts."""
    g = torch.Generator().manual_seed(seed)
    room = prompt + (steps + 1) * 16
    drafter = Drafter(requests, requests * -(-room // page_size), page_size, room,
                      cache_dtype=cache_dtype, seed=seed, device=device)
    lens = torch.randint(1, prompt + 1, (requests,), generator=g).tolist()
    drafter.prompts([torch.randint(drafter.mask_token, (n,), generator=g).to(device) for n in lens])
    last = torch.randint(drafter.mask_token, (requests,), generator=g).to(device)
    tokens, scores = [], []
    for step in range(steps):
        t0 = time.perf_counter()
        drafted, score = drafter.draft(last)
        taken = torch.randint(1, drafter.S + 1, (requests,), generator=g).to(device)
        last = drafted.gather(1, taken[:, None] - 1)[:, 0].long()
        drafter.take(taken)
        tokens.append(drafted)
        scores.append(score)
        if show:
            torch.cuda.synchronize()
            print(f"step {step}: {1e3 * (time.perf_counter() - t0):.2f} ms, contexts "
                  f"{drafter.context.tolist()}, request 0 drafts {drafted[0].tolist()}")
    check_status()
    return torch.stack(tokens), torch.stack(scores)


def main() -> None:
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--requests", type=int, default=8)
    a.add_argument("--prompt", type=int, default=400, help="longest prompt")
    a.add_argument("--steps", type=int, default=4)
    a.add_argument("--page-size", type=int, default=16)
    a.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    a = a.parse_args()
    run(a.requests, a.prompt, a.steps, a.page_size,
        torch.float8_e4m3fn if a.cache == "e4m3" else torch.bfloat16, show=True)


if __name__ == "__main__":
    main()
