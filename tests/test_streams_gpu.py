"""Calls on a stream that is not the current one: what a call allocates belongs to that stream, and
results do not depend on what the current stream does meanwhile."""

from __future__ import annotations

import pytest
import torch

import paged
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
    """name -> (inputs, call(stream, ...)) of every entry point that launches work."""
    g = torch.Generator().manual_seed(0)
    R, S, V, H, K, rank = 3, 4, 4096, 256, 4, 64
    bf = lambda *shape: torch.randn(shape, generator=g).to(BF).to(dev)          # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)             # noqa: E731
    logits = torch.randn((R, S, V), generator=g).to(dev)
    hidden, head, proj, pred, succ = bf(R, S, H), bf(V, H), bf(rank, H), bf(V, rank), bf(V, rank)
    anchors = i32(5, 6, 7)
    ids, unary, h, edges = ds.dflash_selector(logits, hidden, proj, pred, succ, anchors, K)
    b = paged.Batch([20011, 9000, 3], [1, 16, 2], 8, 2, 128, 64, seed=9)
    # tables: the second half of each row is new in every call
    ctx, new, held, free = i32(30, 5, 64), i32(40, 9, 1), i32(2, 1, 4), i32(*range(100, 140))
    table = torch.arange(30, dtype=torch.int32, device=dev).reshape(3, 10).contiguous()
    return {
        "topk": lambda **s: ds.dflash_topk_candidates(logits, K, **s),
        "lmhead_topk": lambda **s: ds.dflash_lmhead_topk(hidden, head, K, **s),
        "projection": lambda **s: (ds.dflash_hidden_projection(hidden, proj, **s),),
        "edges": lambda **s: (ds.dflash_candidate_edges(pred, succ, ids, unary, h, anchors, **s),),
        "selector": lambda **s: ds.dflash_selector(logits, hidden, proj, pred, succ, anchors, K, **s),
        "forward": lambda **s: ds.dflash_selector_forward(ids, unary, hidden, anchors, proj, pred,
                                                          succ, **s),
        "selector_lmhead": lambda **s: ds.dflash_selector_lmhead(hidden, head, proj, pred, succ,
                                                                 anchors, K, **s),
        "best_path": lambda **s: ds.dflash_best_path(edges, ids, **s),
        "tables": lambda **s: ds.dflash_block_tables(ctx, new, held, free, table, 16, 50, **s),
        "tables, some given": lambda **s: ds.dflash_block_tables(
            ctx, new, held, free, table, 16, 50, positions=i32(*[0] * 50), **s),
        "attention": lambda **s: ds.dflash_paged_attention(*b.args(), **s),
    }


NAMES = ["topk", "lmhead_topk", "projection", "edges", "selector", "forward", "selector_lmhead",
         "best_path", "tables", "tables, some given", "attention"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream(dev, name, monkeypatch):
    """Outputs and workspaces come from the memory of the stream passed; what is returned is also
    kept until the current stream's work is done."""
    call = calls(dev)[name]
    want = call()
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
    given = 1 if name == "tables, some given" else 0
    assert sum(t.untyped_storage().data_ptr() not in kept for t in got) == given
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_may_allocate_meanwhile(dev, name):
    """The call waits behind other work on its stream while the current stream takes blocks of all
    the sizes that the call has dropped, and writes to them."""
    call = calls(dev)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    nbytes = [1 << k for k in range(9, 27)]
    if name == "attention":
        nbytes += 3 * [ds.dflash_paged_attention_workspace_bytes(3, 19, 8, 2, 128)]
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


def test_any_object_with_a_stream_handle(dev):
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    call = calls(dev)["attention"]
    want, s = call(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=Handle(s))
    s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_the_current_stream_by_name(dev, monkeypatch):
    """The current stream passed as `stream` is no other stream: nothing is switched or recorded."""
    call, s = calls(dev)["attention"], torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()

    def refuse(*a, **k):
        raise AssertionError("the call switched streams")

    with torch.cuda.stream(s):
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "stream", refuse)
            m.setattr(torch.cuda, "set_stream", refuse)
            m.setattr(torch.Tensor, "record_stream", refuse)
            got = call(stream=s)
    got2 = call(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for g, g2, w in zip(got, got2, want):
        assert torch.equal(g, w) and torch.equal(g2, w)


@pytest.mark.parametrize("name", ["selector", "attention", "tables"])
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
