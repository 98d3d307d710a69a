"""Drawn paths and the verification of drafts on the GPU against the 64-bit forms (tests/step.py)."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import step
import draft_candidate_selector_gb300 as ds

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    ds.dflash_device_status(clear=True)
    return d


def clean():
    assert ds.dflash_device_status(clear=True) == 0


def each(t, R):
    """Temperatures of R requests as a list."""
    return t.tolist() if isinstance(t, torch.Tensor) else [t] * R


# ----------------------------------------------------------------------------- drawn paths

def check_path(edges, ids, u, t):
    """fp32 probabilities: expf is within 2^-23, its product with the exponent's lower part 2^-24, in
    the value and in the sum; five additions and a quotient: 12 * 2^-24 of the value at most; below
    2^-126 they may be 0."""
    got = ds.dflash_sample_path(edges, ids, u, temperature=t)
    path, probs = step.sample_path(edges, u, each(t, len(edges)))
    np.testing.assert_array_equal(got[0].cpu().numpy(), path)
    want = np.take_along_axis(ids.cpu().numpy(), path[:, :, None], 2)[:, :, 0]
    np.testing.assert_array_equal(got[1].cpu().numpy(), want)
    err = np.abs(got[2].cpu().double().numpy() - probs)
    assert (err <= 2.0 ** -20 * probs + 2.0 ** -126).all(), float((err / (probs + 1e-300)).max())
    clean()
    return got


def path_inputs(dev, R, S, K, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    edges = spread * torch.randn((R, S, K, K), generator=g)
    ids = torch.randint(0, 2 ** 31 - 1, (R, S, K), generator=g, dtype=torch.int32)
    u = torch.rand((R, S), generator=g)
    t = 0.4 + torch.rand(R, generator=g)
    return edges.to(dev), ids.to(dev), u.to(dev), t.to(dev)


@pytest.mark.parametrize("R,S,K", [(1, 1, 1), (1, 4, 2), (3, 7, 3), (40, 15, 8), (5, 15, 31), (300, 5, 32),
                                   (2, 256, 32), (2, 100, 5), (9, 8, 16), (700, 9, 4), (3, 33, 17)])
def test_paths(dev, R, S, K):
    for spread in (0.01, 2.0, 30.0):
        edges, ids, u, t = path_inputs(dev, R, S, K, R + S, spread)
        check_path(edges, ids, u, t)
        check_path(edges, ids, u, 1.0)


def test_path_borders(dev):
    """Equal scores and numbers that are exactly borders: the candidate behind the border."""
    for K in (2, 4, 8, 16, 32):
        edges = torch.full((1, K, K, K), 3.25, device=dev)
        ids = torch.arange(K, dtype=torch.int32, device=dev).expand(1, K, K).contiguous()
        u = (torch.arange(K, device=dev) / K)[None].contiguous()
        got = check_path(edges, ids, u, 0.7)
        assert got[0][0].tolist() == list(range(K))


def test_path_near_borders(dev):
    """Numbers within a few steps of fp32 of a border, from both sides."""
    edges, ids, u, _ = path_inputs(dev, 400, 1, 32, 5, 1.0)
    _, probs = step.sample_path(edges, u, [1.0] * 400)
    border = np.cumsum(probs[:, 0], 1)[np.arange(400), np.arange(400) % 31]
    near = border.astype(np.float32).view(np.int32) + (np.arange(400) // 31) % 9 - 4
    u = torch.from_numpy(near.astype(np.int32).view(np.float32))[:, None].to(dev)
    check_path(edges, ids, u.contiguous(), 1.0)


def test_path_greedy_and_odd_rows(dev):
    """Temperatures 0, below, NaN and infinite; rows with NaN and infinities; numbers outside [0, 1)."""
    edges, ids, u, _ = path_inputs(dev, 12, 3, 6, 1)
    edges[:, :, :, 2] = edges[:, :, :, 4]                           # ties
    check_path(edges, ids, u, 0.0)
    t = torch.tensor([0.0, -1.0, NAN, INF, 1e-30, 1e30, 1e-42, 3e38, 1.0, 0.5, 2.0, 1.0], device=dev)
    check_path(edges, ids, u, t)
    edges[0] = NAN
    edges[1] = -INF
    edges[2, :, :, 1] = NAN
    edges[3, :, :, 3] = INF
    edges[4, :, :, 0] = -INF
    edges[5, :, :, 2:] = -INF
    edges[6, :, :, 4] = -3.4e38
    edges[7, :, :, 0] = 3.4e38
    edges[8] = 0.0
    edges[8, :, :, ::2] = -0.0
    edges[9, :, :, :3] = NAN
    edges[9, :, :, 3:] = -INF
    edges[10] = -3.4e38
    for temp in (1.0, 0.0, t):
        check_path(edges, ids, u, temp)
    u[:6] = torch.tensor([NAN, -1.0, 0.0, 1.0, 7.0, INF], device=dev)[:, None]
    check_path(edges, ids, u, 1.0)


def test_path_slices_and_outputs(dev):
    """Slices of requests out of larger arrays (4-byte alignment), and outputs of the caller's own."""
    edges, ids, u, t = path_inputs(dev, 9, 5, 7, 3)
    want = ds.dflash_sample_path(edges, ids, u, temperature=t)
    own = [torch.full_like(x[3:8], -7) for x in want]
    got = ds.dflash_sample_path(edges[3:8], ids[3:8], u[3:8], temperature=t[3:8], path=own[0], tokens=own[1],
                                probs=own[2])
    for g, w, o in zip(got, want, own):
        assert g is o and torch.equal(g, w[3:8])
    clean()


# ----------------------------------------------------------------------------- verification

class Batch:
    """R requests of 0 or more rows; drafts from K likely tokens (K = 0: certain ones)."""

    def __init__(self, dev, rows, V, S=None, K=4, dtype=F32, seed=0, spread=2.0, likely=True, pad_t=0, pad_v=0,
                 offset=0, t=1.0):
        g = torch.Generator().manual_seed(seed)
        R, self.V, self.K, self.t = len(rows), V, K, t
        S = max(0, max(rows) - 1) if S is None else S
        T = sum(rows) + pad_t
        x = spread * torch.randn((T, V), generator=g)
        n = max(K, 1)
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32)
        ids = torch.zeros((R, S, n), dtype=torch.int32)
        probs = torch.zeros((R, S, n))
        drafts = torch.zeros((R, S), dtype=torch.int32)
        for r in range(R):
            for i in range(S):
                c = torch.randperm(V, generator=g)[:n] if V >= n else torch.randint(0, V, (n,), generator=g)
                ids[r, i] = c.to(torch.int32)
                if i < rows[r] - 1:
                    row = int(self.start[r]) + i
                    if likely:
                        x[row, c] = x[row].logsumexp(0) + torch.randn(n, generator=g)
                    probs[r, i] = torch.softmax(x[row, c] + 0.5 * torch.randn(n, generator=g), 0)
                    drafts[r, i] = c[int(torch.multinomial(probs[r, i], 1, generator=g))]
        room = torch.zeros((T, V + pad_v + offset), dtype=dtype)
        room[:, offset:offset + V] = x.to(dtype)
        if pad_v + offset:
            room[:, :offset] = room[:, offset + V:] = NAN                # never read
        if pad_t:
            room[T - pad_t:] = NAN
        self.logits = room.to(dev)[:, offset:offset + V]
        if pad_v + offset == 0:
            self.logits = self.logits.contiguous()
        self.start = self.start.to(dev)
        self.drafts = drafts.to(dev)
        self.ids, self.probs = (ids.to(dev), probs.to(dev)) if K else (None, None)
        self.accept = torch.rand((R, S), generator=g).to(dev)
        self.sample = torch.rand(R, generator=g).to(dev)

    def args(self):
        return (self.logits, self.start, self.drafts, self.accept, self.sample, self.ids, self.probs)

    def run(self, **kw):
        return ds.dflash_verify_drafts(*self.args(), temperature=self.t, **kw)

    def want(self):
        return step.verify(*self.args(), each(self.t, len(self.sample)))

    def check(self, got=None, status=0):
        """Tokens exactly. Log-probabilities: the row's sum is within 2^-17 of itself (its logarithm
        within that), the exponent and the difference are rounded four times."""
        got = self.run() if got is None else got
        tokens, counts, logprobs = self.want()
        np.testing.assert_array_equal(got[0].cpu().numpy(), tokens)
        np.testing.assert_array_equal(got[1].cpu().numpy(), counts)
        err = np.abs(got[2].cpu().double().numpy() - logprobs)
        assert (err <= 2.0 ** -17 + 2.0 ** -22 * np.abs(logprobs)).all(), float(err.max())
        assert ds.dflash_device_status(clear=True) == status
        return got


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 1000, 2047, 2048, 2049, 4096, 4103, 8192, 20011])
def test_vocabularies(dev, V, dtype):
    """Rows of every alignment, shorter than a vector and around the ends of tiles."""
    for K in (0, min(5, V)):
        Batch(dev, [3, 1, 4, 2, 6], V, K=K, dtype=dtype, seed=V).check()


@pytest.mark.parametrize("rows,S", [([1], 0), ([1, 1, 1], 0), ([0, 2, 0, 5, 1, 0], 4), ([16] * 9, 15), ([2], 15),
                                    ([256, 3], 255), ([40, 1], 60), ([0, 0], 3)])
def test_requests(dev, rows, S):
    for K in (0, 3):
        Batch(dev, rows, 700, S, K, seed=len(rows), pad_t=3).check()


@pytest.mark.parametrize("K", [1, 2, 31, 32])
def test_candidates(dev, K):
    Batch(dev, [8] * 20, 5003, K=K, dtype=BF, seed=K).check()


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("pad_v,offset", [(0, 1), (5, 3), (1, 0), (64, 8)])
def test_strided_rows(dev, dtype, pad_v, offset):
    """Rows out of a wider tensor whose other columns and last rows are NaN."""
    Batch(dev, [4, 2, 7], 6001, dtype=dtype, pad_v=pad_v, offset=offset, pad_t=2, seed=offset).check()


@pytest.mark.parametrize("spread", [0.0, 0.01, 0.5])
@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_flat_rows(dev, spread, dtype):
    """Nearly equal logits: borders so close together that fp32 sums do not settle the token."""
    for K in (0, 8):
        Batch(dev, [3] * 30, 50021, K=K, dtype=dtype, spread=spread, seed=3, likely=False).check()


def test_borders(dev):
    """Equal logits and numbers that are exactly borders: the token behind the border; drafts whose
    number is exactly p / q are not taken, one step below they are."""
    V = 2048
    for dtype in (F32, BF):
        b = Batch(dev, [1] * 64, V, 0, 0, dtype)
        b.logits.fill_(-1.5)
        at = torch.arange(64, device=dev) * 32 + 5
        b.sample = at / V
        assert torch.equal(b.check()[0][:, 0].long(), at)
        b = Batch(dev, [2] * 40, V, 1, 0, dtype)
        b.logits.fill_(2.0)
        b.accept = torch.full((40, 1), 1 / V, device=dev)
        b.accept[::2] *= 1 - 2.0 ** -24
        b.drafts = torch.randint(0, V, (40, 1), dtype=torch.int32, device=dev)
        got = b.check()
        assert got[1].tolist() == [2, 1] * 20
        b = Batch(dev, [2] * 40, V, 1, 2, dtype)                      # q = 1/2: p / q = 2 / V
        b.logits.fill_(2.0)
        b.probs.fill_(0.5)
        b.accept = torch.full((40, 1), 2 / V, device=dev)
        b.accept[1::2] *= 1 - 2.0 ** -24
        b.drafts = b.ids[:, :, 1].contiguous()
        assert b.check()[1].tolist() == [1, 2] * 20


def test_near_borders(dev):
    """Numbers within a few steps of fp32 of p / q, and of a border of the row's running sum."""
    b = Batch(dev, [2] * 200, 3001, 1, 4, seed=4)
    p = [step.target(b.logits[2 * r], 1.0) for r in range(200)]
    q = [float(b.probs[r, 0][b.ids[r, 0] == b.drafts[r, 0]].double().sum()) for r in range(200)]
    ratio = np.array([min(0.999, p[r][int(b.drafts[r, 0])] / q[r]) for r in range(200)], np.float32)
    near = ratio.view(np.int32) + np.arange(200) % 9 - 4
    b.accept = torch.from_numpy(near.astype(np.int32).view(np.float32))[:, None].to(dev).contiguous()
    b.check()
    b = Batch(dev, [1] * 300, 3001, 0, 0, seed=5)
    border = np.array([np.cumsum(step.target(b.logits[r], 1.0))[(37 * r) % 2900] for r in range(300)], np.float32)
    near = border.view(np.int32) + np.arange(300) % 9 - 4
    b.sample = torch.from_numpy(near.astype(np.int32).view(np.float32)).clamp(0, 1 - 2 ** -24).to(dev)
    b.check()


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_temperatures(dev, dtype):
    t = torch.tensor([0.0, -1.0, NAN, INF, 1e-30, 1e30, 0.3, 2.5, 1e-3, 1.0], device=dev)
    for K in (0, 4):
        b = Batch(dev, [5] * 10, 9001, K=K, dtype=dtype, seed=8, t=t)
        b.check()
        b.t = 0.0
        b.check()


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_low_temperatures_and_large_logits(dev, dtype):
    """Largest logits of up to 2^70 temperatures, where a product with 1 / T is many units off."""
    t = torch.tensor([10.0 ** -k for k in range(20)], device=dev)
    for K in (0, 4):
        b = Batch(dev, [4] * 20, 5003, K=K, dtype=dtype, seed=9, t=t)
        b.check()
        if dtype != FP:
            b.logits.mul_(10.0 ** 6)
            b.t = t * 10.0 ** 7
            b.check()


def test_greedy_ties(dev):
    """The first of equal largest logits, in the same tile and in a later one; -0 equals +0."""
    b = Batch(dev, [3] * 6, 9000, K=0, t=0.0)
    b.logits.clamp_(max=-0.5)
    for row, at in ((0, (5, 9)), (3, (100, 2100)), (6, (8999,)), (9, (0, 8999)), (12, (2047, 2048)), (15, (3, 4))):
        for k, v in enumerate(at):
            b.logits[row, v] = 0.0 if (k + row) % 2 else -0.0
    b.drafts[:, 0] = torch.tensor([9, 100, 8999, 0, 2048, 3], device=dev)
    got = b.check()
    assert got[0][:, 0].tolist() == [5, 100, 8999, 0, 2047, 3]


def test_masked_logits(dev):
    """Tokens masked by -inf and by the type's lowest value, whole tiles of them, rows with one token or
    none but lowest ones left."""
    for dtype in (F32, BF, FP):
        lowest = torch.finfo(dtype).min
        for mask in (-INF, lowest):
            b = Batch(dev, [3] * 8, 10007, K=4, dtype=dtype, seed=2)
            keep = torch.zeros(10007, dtype=torch.bool, device=dev)
            keep[4000:4400] = True
            keep[torch.arange(0, 10007, 1009, device=dev)] = True
            keep[b.ids.flatten().long()] = True
            b.logits[:, ~keep] = mask
            b.logits[4] = mask
            b.logits[4, 9001] = -7.0
            b.check()
            b.t = 0.0
            b.check()
        b = Batch(dev, [1] * 5, 10007, 0, 0, dtype)
        b.logits.fill_(lowest)
        b.check()


def test_rows_without_a_distribution(dev):
    """NaN, +inf, nothing but -inf: the request ends without a token where such a row is reached, and
    is as it was where it is not."""
    for bad in (NAN, INF, -INF):
        for t in (1.0, 0.0):
            b = Batch(dev, [6] * 12, 5001, K=0, seed=9, t=t)
            b.drafts[::2, 1] = (b.drafts[::2, 1] + 1) % 5001
            first = b.want()[1]
            for r in range(12):
                row = int(b.start[r]) + r % 6
                if bad == -INF:
                    b.logits[row] = bad
                else:
                    b.logits[row, 17 * r] = bad
            reached = [r % 6 < first[r] for r in range(12)]
            assert any(reached) and not all(reached)
            got = b.check(status=ds.DEVICE_BAD_LOGITS)
            for r in range(12):
                assert int(got[1][r]) == (r % 6 if reached[r] else first[r])


def test_bad_tokens(dev):
    """Drafts and candidates outside the vocabulary; a candidate that occurs twice."""
    b = Batch(dev, [4] * 10, 3000, K=4, seed=12)
    b.drafts[2, 0] = -1
    b.drafts[5, 1] = 3000
    b.drafts[7, 0] = 2 ** 31 - 1
    b.check(status=ds.DEVICE_BAD_ID)
    b = Batch(dev, [4] * 10, 3000, K=0, seed=12)
    b.drafts[4, 0] = -5
    b.check(status=ds.DEVICE_BAD_ID)
    b = Batch(dev, [2] * 10, 3000, K=4, seed=12)
    b.accept.fill_(1 - 2.0 ** -24)
    b.logits[::2] += 0.0
    b.ids[:, :, 2] = b.ids[:, :, 0]                                    # the sum of both
    b.check()
    b.ids[3, 0, 1] = -1
    b.ids[4, 0, 3] = 3000
    want = b.want()[1]
    b.check(status=ds.DEVICE_BAD_ID if (want[3] == 1 or want[4] == 1) else 0)


def test_little_left_over(dev):
    """The draft's distribution is nearly, or exactly, the target's: what is left is tiny or nothing."""
    for noise in (0.0, 1e-6, 1e-4):
        b = Batch(dev, [2] * 60, 8, 1, 8, spread=1.0, likely=False, seed=21)
        p = torch.softmax(b.logits[::2].double(), 1)
        b.ids = torch.arange(8, dtype=torch.int32, device=dev).expand(60, 1, 8).contiguous()
        q = p * (1 + noise * torch.randn(60, 8, device=dev).double())
        b.probs = (q / q.sum(1, keepdim=True)).float()[:, None].contiguous()
        b.accept.fill_(1 - 2.0 ** -24)
        b.drafts = (torch.arange(60, device=dev) % 8).to(torch.int32)[:, None].contiguous()
        b.check()


def test_uniforms_outside(dev):
    b = Batch(dev, [1] * 8, 4000, 0, 0)
    b.logits[:, -50:] = -INF
    b.sample = torch.tensor([NAN, -3.0, 0.0, 1.0, 9.0, INF, -INF, 1 - 2.0 ** -24], device=dev)
    got = b.check()
    assert got[0][:3, 0].tolist() == [0, 0, 0] and (got[0][3:6, 0] < 3950).all()


def test_bad_lengths(dev):
    """Rows out of order, before 0, past T, more than S + 1: those requests are refused, not the others."""
    b = Batch(dev, [3, 3, 3, 3], 500, K=3)
    for change in ({2: 2}, {1: -4}, {4: 13}, {0: -1}, {3: 2 ** 31 - 1}, {2: -2 ** 31}):
        c = Batch(dev, [3, 3, 3, 3], 500, K=3)
        for at, v in change.items():
            c.start[at] = v
        c.check(status=ds.DEVICE_BAD_LENGTH)
    c = Batch(dev, [3, 3, 3, 3], 500, 1, K=3)
    c.check(status=ds.DEVICE_BAD_LENGTH)
    clean()


@pytest.mark.parametrize("dtype,V,R,S,K", [(BF, 32768, 100, 15, 8), (F32, 32768, 64, 15, 0), (FP, 30011, 130, 11, 4),
                                           (BF, 151936, 40, 7, 5), (BF, 32768, 250, 15, 8), (FP, 30011, 400, 11, 4),
                                           (BF, 151936, 40, 12, 5)])
def test_large_batches(dev, dtype, V, R, S, K):
    """Batches that pass over rows behind a surely rejected draft, ragged ones too."""
    g = np.random.default_rng(R)
    for rows in ([S + 1] * R, g.integers(0, S + 2, R).tolist()):
        b = Batch(dev, [1] * R, 64, S, 0)                             # numbers only
        T = sum(rows)
        b.V = V
        b.start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=dev)
        gen = torch.Generator(device=dev).manual_seed(R)
        x = 2 * torch.randn((T, V), generator=gen, device=dev)
        n = max(K, 1)
        ids = torch.randint(0, V // n, (R, S, n), generator=gen, device=dev) * n + torch.arange(n, device=dev)
        for r in range(R):
            for i in range(rows[r] - 1):
                x[int(b.start[r]) + i, ids[r, i]] = 14 + torch.randn(n, generator=gen, device=dev)
        b.logits = x.to(dtype)
        b.ids, b.probs = (ids.to(torch.int32), torch.full((R, S, n), 1 / n, device=dev)) if K else (None, None)
        b.drafts = ids[:, :, 0].to(torch.int32).contiguous()
        got = b.check()
        assert 1 < float(got[1].float().mean()) < S
        again = b.run()
        for x, y in zip(got, again):
            assert torch.equal(x, y)


def test_no_rows(dev):
    """No tokens at all: nothing is read."""
    b = Batch(dev, [0, 0, 0], 100, 4, K=3, pad_t=1)
    got = ds.dflash_verify_drafts(b.logits[:0], *b.args()[1:])
    assert (got[0] == -1).all() and not got[1].any() and not got[2].any()
    clean()


def test_the_largest_vocabulary(dev):
    b = Batch(dev, [2, 3, 1], 2 ** 20, K=4, spread=1.0, seed=6)
    b.check()
    b = Batch(dev, [1] * 3, 2 ** 20, 0, 0, BF, spread=0.01, seed=7)
    b.check()
    clean()


def test_rows_past_2_to_the_31_elements(dev):
    """Logits of more than 2^31 elements: the last requests' rows."""
    V = 262144
    T = 2 ** 31 // V + 40
    if torch.cuda.mem_get_info(dev)[0] < 8 * 2 ** 30:
        pytest.skip("needs 8 GB of device memory")
    b = Batch(dev, [4] * 8, V, K=0, dtype=BF, spread=1.0)
    small = b.check()
    far = torch.empty((T, V), dtype=BF, device=dev)
    far[T - 32:] = b.logits
    b.logits, b.start = far, b.start + (T - 32)
    got = b.run()
    for x, y in zip(got, small):
        assert torch.equal(x, y)
    clean()


def test_first_tokens_follow_the_target(dev):
    """Drafts drawn by dflash_sample_path and verified: the first token's frequencies are the target's.
    200000 draws: five standard deviations of each frequency are at most 5 * sqrt(0.25 / 200000)."""
    R, V = 200000, 6
    g = torch.Generator(device=dev).manual_seed(1)
    logits = torch.randn((1, V), generator=g, device=dev).repeat(2 * R, 1)
    edges = torch.randn((1, 1, 1, 4), generator=g, device=dev).expand(R, 1, 4, 4).contiguous()
    ids = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device=dev).expand(R, 1, 4).contiguous()
    rand = lambda *s: torch.rand(s, generator=g, device=dev)                         # noqa: E731
    _, drafts, probs = ds.dflash_sample_path(edges, ids, rand(R, 1), temperature=0.8)
    start = torch.arange(0, 2 * R + 1, 2, dtype=torch.int32, device=dev)
    tokens, counts, _ = ds.dflash_verify_drafts(logits, start, drafts, rand(R, 1), rand(R), ids, probs,
                                                temperature=1.3)
    p = torch.softmax(logits[0].double() / 1.3, 0)
    seen = torch.bincount(tokens[:, 0].long(), minlength=V).double() / R
    assert (seen - p).abs().max() < 5 * math.sqrt(0.25 / R)
    bonus = tokens[counts == 2, 1].long()
    seen = torch.bincount(bonus, minlength=V).double() / len(bonus)
    assert (seen - p).abs().max() < 5 * math.sqrt(0.25 / len(bonus))
    clean()


# ----------------------------------------------------------------------------- calls

def test_workspaces_and_outputs(dev):
    b = Batch(dev, [4] * 10, 9000, dtype=BF)
    want = b.check()
    need = ds.dflash_verify_drafts_workspace_bytes(10, 40, 9000)
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            b.run(workspace=ws)
    with pytest.raises(ValueError, match="needed"):
        b.run(workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    own = dict(tokens=torch.full_like(want[0], 9), counts=torch.full_like(want[1], 9),
               logprobs=torch.full_like(want[2], 9))
    room = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device=dev)
    got = b.run(workspace=room[:need], **own)
    for g, w, o in zip(got, want, own.values()):
        assert g is o and torch.equal(g, w)
    assert (room[need:] == 0xAB).all()
    clean()


def test_in_graphs(dev):
    """Captured and replayed with other inputs; two graphs that share a workspace, one after the other."""
    a = Batch(dev, [8] * 30, 32768, dtype=BF, seed=1)
    b = Batch(dev, [16] * 90, 32768, K=0, dtype=BF, seed=2, likely=False)     # passes over rows
    ws = torch.empty(ds.dflash_verify_drafts_workspace_bytes(90, 1440, 32768), dtype=torch.uint8, device=dev)
    wants = [[x.clone() for x in c.run()] for c in (a, b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c.run(workspace=ws))
        graphs.append(graph)
    for _ in range(3):
        for graph, out, want in zip(graphs, outs, wants):
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(out, want):
                assert torch.equal(x, y)
    a.sample.copy_(torch.rand_like(a.sample))
    a.accept.copy_(torch.rand_like(a.accept))
    graphs[0].replay()
    a.check(outs[0])


def test_two_streams_at_once(dev):
    batches = [Batch(dev, [9] * 60, 32768, dtype=BF, seed=k) for k in range(2)]
    wants = [b.run() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(10):
        gots = [b.run(stream=s) for b, s in zip(batches, streams)]
        torch.cuda.synchronize()
        for got, want in zip(gots, wants):
            for x, y in zip(got, want):
                assert torch.equal(x, y)
    clean()
