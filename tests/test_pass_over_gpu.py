"""The verification of batches so large that rows behind a surely rejected draft are passed over: every kind of
row and request, against the 64-bit form; graphs, streams and workspaces."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import step
import draft_candidate_selector_gb300 as ds
from test_sampling_gpu import BF, F32, FP, INF, NAN, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    ds.dflash_device_status(clear=True)
    return d


class Large(Batch):
    """A batch made on the GPU: n = max(K, 1) likely tokens a row, drafts among them."""

    def __init__(self, dev, dtype, V, rows, S, K, seed=0, t=1.0):
        R, T, n = len(rows), sum(rows), max(K, 1)
        self.V, self.K, self.t = V, K, t
        g = torch.Generator(device=dev).manual_seed(seed)
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=dev)
        x = 2 * torch.randn((T, V), generator=g, device=dev)
        ids = torch.randint(0, V // n, (R, S, n), generator=g, device=dev) * n + torch.arange(n, device=dev)
        of = torch.repeat_interleave(torch.arange(R, device=dev), torch.tensor(rows, device=dev))
        at = torch.arange(T, device=dev) - self.start[:-1].long()[of]
        drafted = at < torch.clamp(self.start[1:] - self.start[:-1] - 1, max=S)[of]
        rows_at = drafted.nonzero()[:, 0]
        lift = 14 + torch.randn((len(rows_at), n), generator=g, device=dev)
        x[rows_at[:, None], ids[of[rows_at], at[rows_at]]] = lift
        self.logits = x.to(dtype)
        self.ids, self.probs = None, None
        if K:
            self.ids, self.probs = ids.to(torch.int32), torch.full((R, S, n), 1 / n, device=dev)
        self.drafts = ids[:, :, 0].to(torch.int32).contiguous()
        self.accept = torch.rand((R, S), generator=g, device=dev)
        self.sample = torch.rand(R, generator=g, device=dev)

    def workspace(self, fill=0, more=0):
        R, S = self.drafts.shape
        T, V = self.logits.shape
        need = ds.dflash_verify_drafts_workspace_bytes(R, T, V)
        return torch.full((need + more,), fill, dtype=torch.uint8, device=self.logits.device)[:need]

    def tiles(self):
        """Tiles of 4 KB in all rows."""
        T, V = self.logits.shape
        return T * -(-V * self.logits.element_size() // 4096)

    def check_passing(self, status=0, least=1):
        """Results as the 64-bit form's; and that this batch is of those that pass rows over, which start from
        sums that are all ones. (Where every row is read, no word of a workspace becomes that.)"""
        ws = self.workspace()
        got = self.check(self.run(workspace=ws), status)
        left = int((ws.view(torch.int64) == -1).sum())
        assert left >= least, (left, least)
        return got


# Rows of 11, 5 and 3 pieces of 32 KB, found by fours, threes and twos, the last group of a row shorter.
SIZES = [(F32, 90001, 200, 3, 0), (F32, 90001, 200, 3, 5), (BF, 70001, 300, 3, 4), (BF, 70001, 300, 3, 0),
         (FP, 40011, 400, 11, 4)]


@pytest.mark.parametrize("dtype,V,R,S,K", SIZES)
def test_rows_without_a_distribution(dev, dtype, V, R, S, K):
    """NaN, +inf or nothing but -inf before, at and behind the first rejected draft, in any tile."""
    b = Large(dev, dtype, V, [S + 1] * R, S, K, seed=V)
    first = b.want()[1]
    g = np.random.default_rng(R)
    reached = 0
    for r in range(0, R, 2):
        i, row = int(g.integers(0, S + 1)), int(b.start[r])
        reached += i < first[r]
        bad = (NAN, INF, -INF)[r // 2 % 3]
        if bad == -INF:
            b.logits[row + i] = bad
        else:
            b.logits[row + i, int(g.integers(0, V))] = bad
    assert 0 < reached < R // 2
    b.check_passing(status=ds.DEVICE_BAD_LOGITS)


@pytest.mark.parametrize("dtype,V,R,S,K", SIZES)
def test_requests_and_temperatures(dev, dtype, V, R, S, K):
    """Requests of every length, none and too many rows among them; a temperature for each, greedy ones among
    them; drafts that are no tokens."""
    g = np.random.default_rng(V)
    rows = g.integers(0, S + 2, R)
    rows[5::40] = S + 2
    rows[3::40] = S + 1
    t = torch.from_numpy(g.choice([0.0, 1.0, 0.7, 1.4, -1.0, 1e-3, 30.0], R).astype(np.float32)).to(dev)
    b = Large(dev, dtype, V, rows.tolist(), S, K, seed=R, t=t)
    b.drafts[3::40, 0] = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31], device=dev).repeat(R)[
        :len(b.drafts[3::40])].to(torch.int32)
    b.drafts[6::40, S - 1] = V + 7
    b.check_passing(status=ds.DEVICE_BAD_LENGTH | ds.DEVICE_BAD_ID)


@pytest.mark.parametrize("dtype,V,R,S,K", SIZES)
def test_greedy_ties(dev, dtype, V, R, S, K):
    """The first of equal largest logits: drafts that are that one, a later one, or none."""
    b = Large(dev, dtype, V, [S + 1] * R, S, 0, seed=V + 1, t=0.0)
    g = np.random.default_rng(R)
    rows, width = R * (S + 1), V - 1
    a = torch.from_numpy(g.integers(0, width, rows)).to(dev)
    z = torch.from_numpy(g.integers(0, width, rows)).to(dev)
    every = torch.arange(rows, device=dev)
    b.logits[every, a] = 20.0
    b.logits[every, z] = 20.0
    low, high = torch.minimum(a, z).view(R, S + 1), torch.maximum(a, z).view(R, S + 1)
    which = torch.from_numpy(g.random((R, S + 1))).to(dev)
    drafts = torch.where(which < 0.7, low, torch.where(which < 0.85, high, torch.full_like(low, V - 1)))
    b.drafts = drafts[:, :S].to(torch.int32).contiguous()
    got = b.check_passing()
    assert 1 < float(got[1].float().mean()) < S + 1


def test_which_batches(dev):
    """A small batch reads all of its rows."""
    b = Large(dev, BF, 32768, [4] * 20, 3, 2)
    ws = b.workspace()
    b.check(b.run(workspace=ws))
    assert not (ws.view(torch.int64) == -1).any()
    Large(dev, BF, 32768, [16] * 250, 15, 2).check_passing()


def test_workspaces(dev):
    """What a workspace holds on entry does not matter, and nothing behind it is written."""
    b = Large(dev, BF, 70001, [4] * 300, 3, 4, seed=1)
    want = b.check_passing()
    for fill in (0xFF, 0x7F, 0x00, 0x80):
        ws = b.workspace(fill, 4096)
        for x, y in zip(b.run(workspace=ws), want):
            assert torch.equal(x, y)
        room = ws.as_strided((len(ws) + 4096,), (1,))
        assert (room[len(ws):] == fill).all()
    assert ds.dflash_device_status(clear=True) == 0


def test_in_graphs(dev):
    """Two captured batches that share a workspace, replayed in turn and on other numbers."""
    batches = [Large(dev, BF, 32768, [16] * 250, 15, 8, seed=2), Large(dev, F32, 90001, [4] * 200, 3, 0, seed=3)]
    wants = [[x.clone() for x in b.check_passing()] for b in batches]
    ws = max((b.workspace() for b in batches), key=len)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in batches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(b.run(workspace=ws))
        graphs.append(graph)
    for _ in range(3):
        for graph, out, want in zip(graphs, outs, wants):
            for x in out:
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(out, want):
                assert torch.equal(x, y)
    for graph, out, b in zip(graphs, outs, batches):
        b.accept.copy_(torch.rand_like(b.accept))
        b.sample.copy_(torch.rand_like(b.sample))
        graph.replay()
        b.check(out)


def test_two_streams_at_once(dev):
    batches = [Large(dev, BF, 32768, [16] * 250, 15, 8, seed=k) for k in (4, 5)]
    wants = [b.check_passing() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(10):
        gots = [b.run(stream=s) for b, s in zip(batches, streams)]
        torch.cuda.synchronize()
        for got, want in zip(gots, wants):
            for x, y in zip(got, want):
                assert torch.equal(x, y)
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.parametrize("mask", ["-inf", "lowest"])
@pytest.mark.parametrize("dtype,K", [(BF, 0), (BF, 4), (F32, 4), (FP, 4)])
def test_masked_drafts(dev, dtype, K, mask):
    """Drafts that the target masks are surely rejected, and the rows behind them are passed over."""
    R, S, V = 64, 15, 100003
    b = Large(dev, dtype, V, [S + 1] * R, S, K, seed=7)
    low = -INF if mask == "-inf" else torch.finfo(dtype).min
    keep = torch.zeros(V, dtype=torch.bool, device=dev)
    keep[torch.arange(11, V, 1999, device=dev)] = True
    keep[b.ids.flatten().long() if K else b.drafts.flatten().long()] = False
    assert int(keep.sum()) > 20
    b.logits[:, ~keep] = low
    b.accept.clamp_(min=2.0 ** -20)
    got = b.check_passing(least=b.tiles() // 4)
    assert (got[1] == 1).all() and keep[got[0][:, 0].long()].all()
    b.accept[::2] = 0.0                                              # 0 < p does not hold either
    b.check_passing(least=b.tiles() // 4)
    if K:
        b.probs.zero_()
        b.check_passing(least=b.tiles() // 4)
