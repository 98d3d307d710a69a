"""The sampled step's calls on a stream that is not the current one, and captured on one."""

from __future__ import annotations

import pytest
import torch

import draft_candidate_selector_gb300 as ds

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    ds.dflash_device_status(clear=True)
    return d


def calls(dev):
    g = torch.Generator().manual_seed(0)
    R, S, K, V, T = 40, 9, 5, 32768, 300
    rand = lambda *s: torch.rand(s, generator=g).to(dev)                                # noqa: E731
    q, k, v = (torch.randn((T, h, 64), generator=g).to(BF).to(dev) for h in (4, 2, 2))
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    freq = ds.dflash_rope_frequencies(64, device=dev)
    kc, vc = (torch.zeros((20, 16, 2, 64), dtype=BF, device=dev) for _ in range(2))
    slots = torch.randperm(320, generator=g)[:T].to(dev)
    edges = torch.randn((R, S, K, K), generator=g).to(dev)
    ids = torch.randint(0, V, (R, S, K), generator=g, dtype=torch.int32).to(dev)
    u, accept, last = rand(R, S), rand(R, S), rand(R)
    logits = (3 * torch.randn((R * (S + 1), V), generator=g)).to(BF).to(dev)
    start = torch.arange(0, R * (S + 1) + 1, S + 1, dtype=torch.int32, device=dev)
    _, drafts, probs = ds.dflash_sample_path(edges, ids, u)
    w = torch.ones(64, dtype=BF, device=dev)
    return {
        "norm_rope": lambda **s: ds.dflash_qk_norm_rope(q, k, pos, freq, w, w, **s),
        "norm_rope_store": lambda **s: ds.dflash_qk_norm_rope_store(q, k, v, pos, slots, kc, vc, freq, w, w, **s),
        "sample_path": lambda **s: ds.dflash_sample_path(edges, ids, u, **s),
        "verify": lambda **s: ds.dflash_verify_drafts(logits, start, drafts, accept, last, ids, probs, **s),
    }


NAMES = ["norm_rope", "norm_rope_store", "sample_path", "verify"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream(dev, name, monkeypatch):
    """Outputs and workspaces come from the memory of the stream passed, and outputs are kept until the
    current stream's work is done."""
    call = calls(dev)[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    s, seen, recorded = torch.cuda.Stream(), [], []
    empty, record = torch.empty, torch.Tensor.record_stream

    def spy_empty(*a, **k):
        seen.append(torch.cuda.current_stream())
        return empty(*a, **k)

    def spy_record(t, stream):
        recorded.append((t.untyped_storage().data_ptr(), stream))
        return record(t, stream)

    with monkeypatch.context() as m:
        m.setattr(torch, "empty", spy_empty)
        m.setattr(torch.Tensor, "record_stream", spy_record)
        got = call(stream=s)
    s.synchronize()
    assert seen and all(x == s for x in seen)
    assert all(x == torch.cuda.current_stream() for _, x in recorded)
    kept = {at for at, _ in recorded}
    given = 2 if name == "norm_rope_store" else 0                    # the caches
    assert sum(t.untyped_storage().data_ptr() not in kept for t in got) == given
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_may_allocate_meanwhile(dev, name):
    call = calls(dev)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    nbytes = [1 << k for k in range(9, 25)] + 3 * [ds.dflash_verify_drafts_workspace_bytes(40, 400, 32768)]
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)              # about 10 ms
        got = call(stream=s)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) for n in nbytes]
        del junk
        s.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        torch.cuda.synchronize()
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.parametrize("name", NAMES)
def test_another_stream_in_a_graph(dev, name):
    """A call on a stream that a capture has forked to."""
    call = calls(dev)[name]
    want = [t.clone() for t in call()]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    assert ds.dflash_device_status(clear=True) == 0


def test_a_whole_step_in_one_graph(dev):
    """Norm, rotation and store, a drawn path and its verification, captured together and replayed on other
    numbers."""
    c = calls(dev)
    g = torch.Generator(device=dev).manual_seed(5)
    R, S, K, V = 40, 9, 5, 32768
    edges = torch.randn((R, S, K, K), generator=g, device=dev)
    ids = torch.randint(0, V, (R, S, K), generator=g, device=dev, dtype=torch.int32)
    logits = 3 * torch.randn((R * (S + 1), V), generator=g, device=dev)
    start = torch.arange(0, R * (S + 1) + 1, S + 1, dtype=torch.int32, device=dev)
    u = [torch.rand(s, generator=g, device=dev) for s in ((R, S), (R, S), (R,))]

    def run():
        stored = c["norm_rope_store"]()
        path, drafts, probs = ds.dflash_sample_path(edges, ids, u[0], temperature=0.9)
        return stored[:1] + (path, *ds.dflash_verify_drafts(logits, start, drafts, u[1], u[2], ids, probs,
                                                            temperature=0.8))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for x in u:
            x.copy_(torch.rand(x.shape, generator=g, device=dev))
        graph.replay()
        for x, y in zip(got, run()):
            assert torch.equal(x, y)
    assert ds.dflash_device_status(clear=True) == 0
