"""The paged cache operators on the GPU against plain 64-bit forms (tests/paged.py)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import paged
import draft_candidate_selector_gb300 as ds

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


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


# ----------------------------------------------------------------------------- block tables

def run_tables(dev, ctx, new, held, free, table, page, T):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)   # noqa: E731
    t = i32(table)
    got = ds.dflash_block_tables(i32(ctx), i32(new), i32(held), i32(free), t, page, T)
    want = paged.tables(ctx, new, held, free, np.asarray(table), page, T)
    names = ["query_start", "kv_lens", "held", "positions", "slots", "needed"]
    np.testing.assert_array_equal(t.cpu().numpy(), want[0], "block_table")
    for name, g, w in zip(names, got, want[1:7]):
        np.testing.assert_array_equal(g.cpu().numpy().ravel(), np.ravel(w), name)
    return want


def make_tables(seed, R, page, most_ctx, most_new, extra=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, most_ctx + 1, R)
    new = rng.integers(0, most_new + 1, R)
    held = -(-ctx // page) + rng.integers(0, extra + 1, R)
    width = int(max(1, (-(-(ctx + new) // page)).max(), held.max())) + 1
    order = rng.permutation(int(held.sum()) + int((-(-(ctx + new) // page)).sum()) + 3)
    table = np.full((R, width), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    return ctx, new, held, order[at:], table, page, int(new.sum())


@pytest.mark.parametrize("R,page,most_ctx,most_new,extra", [
    (1, 16, 0, 1, 0), (1, 1, 5, 9, 0), (3, 7, 40, 20, 2), (64, 16, 500, 16, 1),
    (255, 16, 100, 3, 0), (256, 64, 300, 200, 3), (257, 5, 33, 11, 0), (1000, 32, 64, 40, 2),
    (16384, 16, 40, 2, 1), (2, 128, 1000, 3000, 0)])
def test_tables(dev, R, page, most_ctx, most_new, extra):
    run_tables(dev, *make_tables(R, R, page, most_ctx, most_new, extra))
    clean()


def test_tables_padded_and_empty(dev):
    """Room for more tokens than there are; no new tokens at all; no room and no tokens."""
    ctx, new, held, free, table, page, T = make_tables(5, 40, 16, 100, 7)
    run_tables(dev, ctx, new, held, free, table, page, T + 133)
    run_tables(dev, ctx, 0 * new, held, free, table, page, 9)
    run_tables(dev, ctx, 0 * new, held, free[:0], table, page, 0)
    clean()


def test_tables_refuse_bad_lengths(dev):
    """A negative length, a context longer than its pages, a row that is too short: refused one
    by one, with the others' results unchanged."""
    ctx, new, held, free, table, page, T = make_tables(6, 20, 8, 100, 30)
    new = new + 1
    T = int(new.sum())
    for r, what in ((3, "ctx"), (7, "new"), (11, "long"), (15, "held")):
        c, n, h = ctx.copy(), new.copy(), held.copy()
        if what == "ctx":
            c[r] = -5
        elif what == "new":
            n[r] = -1
        elif what == "long":
            n[r] = table.shape[1] * page + 1
        else:
            c[r] = h[r] * page + 1
        room = int(np.maximum(n, 0).sum())
        want = run_tables(dev, c, n, h, free, table, page, room)
        assert want[7].tolist() == [i == r for i in range(20)]
        assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_LENGTH


def test_tables_extreme_lengths(dev):
    """Lengths near 2^31: no sum wraps."""
    big = 2 ** 31 - 1
    want = run_tables(dev, [5, big, 3, 0], [0, big, 2, 1], [1, 1, 1, 0], [9, 8],
                      [[4, -1], [5, -1], [6, -1], [-1, -1]], 8, 0)
    assert want[7].tolist() == [False, True, False, False]
    assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_LENGTH


@pytest.mark.parametrize("short", [1, 5, 1000000])
def test_tables_pool_too_short(dev, short):
    ctx, new, held, free, table, page, T = make_tables(7, 30, 16, 100, 90)
    need = int(np.maximum(0, -(-(ctx + new) // page) - held).sum())
    want = run_tables(dev, ctx, new, held, free[:max(0, need - short)], table, page, T)
    assert want[7].any()
    assert ds.dflash_device_status(clear=True) == ds.DEVICE_NO_PAGES


def test_tables_too_little_room(dev):
    ctx, new, held, free, table, page, T = make_tables(8, 12, 16, 100, 30)
    run_tables(dev, ctx, new, held, free, table, page, T - 5)
    assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_LENGTH


# ----------------------------------------------------------------------------- store

def plain_store(x, slots, cache, scale):
    """The cache after the store, on the CPU: rows by slot, e4m3 by an fp32 division and torch's
    own rounding of a clamped value."""
    page = cache.shape[1]
    if cache.dtype == E4:
        x = (x.float() / scale).clamp(-448, 448).to(E4).view(torch.uint8)
        cache = cache.view(torch.uint8)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            cache[s // page, s % page] = x[t]


@pytest.mark.parametrize("dtype,small,layout,T,H,D,page", [
    (BF, False, "nhd", 1, 1, 8, 1), (FP, False, "hnd", 37, 3, 128, 16),
    (BF, True, "nhd", 37, 2, 64, 16), (FP, True, "hnd", 300, 5, 16, 7),
    (BF, False, "nhd", 1000, 8, 256, 64), (BF, True, "hnd", 1000, 8, 128, 128)])
def test_store(dev, dtype, small, layout, T, H, D, page):
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn((T, 4 * H, D), generator=g).to(dtype)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::7] = -1 - slots[::7]
    shape = (pages, H, page, D) if layout == "hnd" else (pages, page, H, D)
    cdt = E4 if small else dtype
    caches = [torch.randn(shape, generator=g).to(cdt) for _ in range(2)]
    ks, vs = (0.3, 0.007) if small else (1.0, 1.0)
    dcaches = [c.to(dev) for c in caches]
    view = (lambda c: c.transpose(1, 2)) if layout == "hnd" else (lambda c: c)   # noqa: E731
    d = qkv.to(dev)
    ds.dflash_store_kv(d[:, H:2 * H], d[:, 3 * H:], slots.to(dev), *map(view, dcaches),
                       k_scale=ks, v_scale=vs)
    plain_store(qkv[:, H:2 * H], slots, view(caches[0]), ks)
    plain_store(qkv[:, 3 * H:], slots, view(caches[1]), vs)
    raw = torch.uint8 if small else torch.int16
    for got, want in zip(dcaches, caches):
        assert torch.equal(got.cpu().view(raw), want.view(raw))
    clean()


def test_store_every_value_to_e4m3(dev):
    """All 2^16 bf16 and fp16 bit patterns, NaN and infinities among them."""
    for dtype, scale in ((BF, 1.0), (FP, 1.0), (BF, 0.3), (FP, 37.0)):
        x = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(dtype)
        x = x.reshape(512, 1, 128)
        c = torch.zeros((32, 16, 1, 128)).to(E4)
        d = [c.to(dev), c.to(dev)]
        slots = torch.arange(512)
        ds.dflash_store_kv(x.to(dev), x.to(dev), slots.to(dev), *d, k_scale=scale, v_scale=scale)
        plain_store(x, slots, c, scale)
        want = c.float()
        for got in d:
            got = got.cpu().float()
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got[~want.isnan()], want[~want.isnan()])


def test_store_bad_slots_and_nothing(dev):
    x = torch.ones((4, 2, 64), dtype=BF, device=dev)
    c = [torch.zeros((3, 16, 2, 64), dtype=BF, device=dev) for _ in range(2)]
    ds.dflash_store_kv(x, x, torch.tensor([-1, 48, 5, 2 ** 40], device=dev), *c)
    assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_ID
    for t in c:
        assert t.sum() == 128 and (t[0, 5] == 1).all()
    ds.dflash_store_kv(x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device=dev), *c)
    clean()


# ----------------------------------------------------------------------------- attention

def check(b, what="", **kw):
    opts = dict(window_left=kw.get("left", -1), window_right=kw.get("right", 0),
                softcap=kw.get("softcap", 0.0), **b.scales())
    if "scale" in kw:
        opts["scale"] = kw["scale"]
    got = ds.dflash_paged_attention(*b.args(), **opts)
    paged.assert_attention(got, paged.attention(b, **kw), what)
    clean()
    return got


# head_dim and page sizes of both kernels: 64 and 128 on pages of 8 to 256 tokens, and others
SHAPES = [(64, 16), (128, 16), (128, 8), (64, 32), (128, 64), (128, 128), (64, 256),
          (8, 16), (80, 16), (256, 16), (128, 1), (64, 7)]
TYPES = [(BF, None), (FP, None), (BF, E4), (FP, E4)]


@pytest.mark.parametrize("D,page", SHAPES)
@pytest.mark.parametrize("dtype,cache", TYPES)
def test_attention_shapes(dev, D, page, dtype, cache):
    if cache is E4 and D % 16:
        D = 16
    b = paged.Batch([0, 5, 130, 300, 63], [3, 1, 9, 20, 64], 4, 2, D, page, dtype, cache, seed=D)
    check(b)
    check(b, right=-1)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 5), (10, 2), (12, 2), (14, 2),
                                    (8, 1), (16, 1), (48, 1), (128, 1), (130, 1)])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_attention_heads(dev, Hq, Hkv, layout):
    b = paged.Batch([0, 40, 200], [1, 17, 150], Hq, Hkv, 128, 16, layout=layout, seed=Hq)
    check(b)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
def test_attention_lengths(dev, n):
    """Lengths on every side of the tiles' edges, cached and new."""
    ctx = [0, 1, 127, 128, 129, 255, 256, 511]
    b = paged.Batch(ctx, [n] * len(ctx), 4, 1, 64, 16, seed=n)
    check(b)
    check(b, right=-1, left=100)


@pytest.mark.parametrize("left,right", [(0, 0), (1, 0), (5, 3), (127, 0), (128, -1), (-1, 7),
                                        (300, 300), (-1, -1), (1000, 0)])
def test_attention_windows(dev, left, right):
    b = paged.Batch([0, 33, 500, 1000], [100, 16, 16, 40], 6, 2, 128, 32, seed=left + 7)
    check(b, left=left, right=right)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("softcap,spread,scale", [(0.0, 6.0, None), (30.0, 6.0, None),
                                                  (2.0, 1.0, 0.3), (50.0, 1.0, 0.01)])
def test_attention_scores(dev, dtype, cache, softcap, spread, scale):
    """Peaked scores, capped scores and scales other than the default."""
    b = paged.Batch([700, 0, 90], [1, 70, 16], 8, 2, 128, 16, dtype, cache, seed=3, spread=spread)
    kw = {} if scale is None else dict(scale=scale)
    check(b, softcap=softcap, **kw)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_attention_long_contexts(dev, dtype, cache, D):
    """Few rows over long contexts, which are split over the chip and joined."""
    b = paged.Batch([20011, 9000, 3], [1, 16, 2], 8, 2, D, 64, dtype, cache, seed=9, spread=3.0)
    check(b)
    check(b, left=6000, right=-1)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_attention_mixed_batch(dev, dtype, cache, D):
    """Single tokens, blocks and prompt chunks in one batch of many requests, in every order, so that
    one SM takes items of all kinds one after another."""
    rng = np.random.default_rng(15)
    new = rng.choice([1, 1, 2, 8, 16, 40, 130, 300], 160)
    ctx = rng.integers(0, 600, 160)
    b = paged.Batch(ctx, new, 4, 1, D, 16, dtype, cache, seed=15)
    want = check(b)
    for _ in range(10):
        for g, w in zip(ds.dflash_paged_attention(*b.args(), **b.scales()), want):
            assert torch.equal(g, w)
    check(b, left=150, right=4, softcap=15.0)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_attention_many_steps(dev, dtype, cache):
    """Single tokens over contexts long enough that each part of a split has many key tiles, from
    pages all over a large pool: right, and the same bits every time."""
    b = paged.Batch([60000, 90001], [1, 1], 4, 1, 128, 16, dtype, cache, seed=14, spread=2.0)
    want = check(b)
    for _ in range(40):
        for g, w in zip(ds.dflash_paged_attention(*b.args(), **b.scales()), want):
            assert torch.equal(g, w)
    clean()


def test_attention_empty_rows(dev):
    """A request with no cached key at all gives zeros and -inf; so does one whose length is less
    than its new tokens, for the tokens in front of it; requests without tokens give nothing."""
    b = paged.Batch([10, 0, 6, 0, 50], [5, 4, 0, 0, 1], 4, 2, 64, 16, seed=1)
    b.kv_lens[1] = 0
    b.kv[1] = 0
    out, lse = check(b)
    assert not out[5:9].any() and torch.isinf(lse[5:9]).all()
    b.kv_lens[1] = 2
    out, lse = ds.dflash_paged_attention(*b.args())
    assert not out[5:7].any() and torch.isinf(lse[5:7]).all()
    assert torch.isfinite(lse[7:9]).all() and torch.isfinite(out).all()
    clean()


@pytest.mark.parametrize("D", [64, 128, 80])
@pytest.mark.parametrize("junk", [float("inf"), float("nan"), -float("inf")])
def test_attention_hidden_values_have_no_effect(dev, D, junk):
    """What rows do not see may be anything: pool rows of nobody and behind the last token (they
    hold junk in every test here), keys and values of later tokens, keys that left the window."""
    b = paged.Batch([200, 3, 0], [40, 16, 150], 4, 2, D, 16, seed=4, junk=junk)
    want = [t.clone() for t in ds.dflash_paged_attention(*b.args(), window_left=50)]
    for r in range(3):                        # the last token's key and value, seen by it alone
        j = int(b.kv[r]) - 1
        page, row = int(b.table[r, j // 16]), j % 16
        b.key_cache[page, row] = junk
        b.value_cache[page, row] = junk
    j = 100                                   # a key that every row's window has left
    b.key_cache[int(b.table[0, j // 16]), j % 16] = junk
    b.value_cache[int(b.table[0, j // 16]), j % 16] = junk
    got = ds.dflash_paged_attention(*b.args(), window_left=50)
    last = torch.tensor([39, 55, 205], device=dev)
    keep = torch.ones(b.T, dtype=torch.bool, device=dev)
    keep[last] = False
    for g, w in zip(got, want):
        assert torch.equal(g[keep], w[keep])
    assert not torch.isfinite(got[0][last]).all()
    clean()


def test_attention_visible_nan_and_infinity(dev):
    """A NaN in a visible key reaches the rows that see it; an infinite value gives infinities."""
    b = paged.Batch([30], [8], 2, 1, 64, 16, seed=5)
    b.value_cache[int(b.table[0, 0]), 3, 0, 5] = float("inf")
    out, lse = ds.dflash_paged_attention(*b.args())
    assert torch.isinf(out[:, :, 5]).all() and torch.isfinite(lse).all()
    assert torch.isfinite(out[:, :, :5]).all() and torch.isfinite(out[:, :, 6:]).all()
    b.key_cache[int(b.table[0, 2]), 1, 0, 0] = float("nan")     # key 33: seen by tokens 3..7
    out, lse = ds.dflash_paged_attention(*b.args())
    assert torch.isnan(out[3:]).all() and torch.isnan(lse[3:]).all()
    assert torch.isfinite(lse[:3]).all()
    clean()


def test_attention_bad_pages(dev):
    """A page id outside the pool is never followed: its request is NaN, the others are right."""
    b = paged.Batch([60, 60, 700], [4, 16, 1], 4, 2, 128, 16, seed=6)
    want = ds.dflash_paged_attention(*b.args())
    for bad in (-1, b.key_cache.shape[0], 2 ** 31 - 1):
        b.block_table[1, 2] = bad
        got = ds.dflash_paged_attention(*b.args())
        assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_ID
        assert torch.isnan(got[0][4:20]).all() and torch.isnan(got[1][4:20]).all()
        for g, w in zip(got, want):
            assert torch.equal(g[:4], w[:4]) and torch.equal(g[20:], w[20:])


def test_attention_bad_lengths(dev):
    b = paged.Batch([60, 60, 700], [4, 16, 1], 4, 2, 128, 16, seed=6)
    want = ds.dflash_paged_attention(*b.args())
    for bad in (-3, b.max_pages * 16 + 1, 2 ** 31 - 1):
        b.kv_lens[1] = bad
        got = ds.dflash_paged_attention(*b.args())
        assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_LENGTH
        assert torch.isnan(got[0][4:20]).all() and torch.isnan(got[1][4:20]).all()
        for g, w in zip(got, want):
            assert torch.equal(g[:4], w[:4]) and torch.equal(g[20:], w[20:])


def test_attention_rows_behind_the_last_request(dev):
    """A padded batch: rows behind query_start[R] are not written."""
    b = paged.Batch([60, 9], [4, 16], 4, 2, 64, 16, seed=6)
    want = ds.dflash_paged_attention(*b.args())
    q = torch.cat([b.query, torch.full((13, 4, 64), float("nan"), dtype=BF, device=dev)])
    out = torch.full((33, 4, 64), 7.0, dtype=BF, device=dev)
    lse = torch.full((33, 4), 7.0, device=dev)
    ds.dflash_paged_attention(q, *b.args()[1:], out=out, lse=lse)
    assert torch.equal(out[:20], want[0]) and torch.equal(lse[:20], want[1])
    assert (out[20:] == 7).all() and (lse[20:] == 7).all()
    clean()


def test_attention_offsets_past_32_bits(dev):
    """Pages behind 2^31 elements of a pool."""
    page, H, D = 64, 4, 128
    skip = 2 ** 31 // (page * H * D) + 10
    b = paged.Batch([500, 0], [3, 70], 8, H, D, page, device="cpu", seed=8)
    big = []
    for c in (b.key_cache, b.value_cache):
        t = torch.zeros((skip + c.shape[0], page, H, D), dtype=BF, device=dev)
        t[skip:] = c.to(dev)
        big.append(t)
    args = (b.query.to(dev), *big, (b.block_table + skip).to(dev), b.query_start.to(dev),
            b.kv_lens.to(dev))
    paged.assert_attention(ds.dflash_paged_attention(*args), paged.attention(b))
    x = torch.randn((5, H, D), device=dev).to(BF)
    slots = torch.arange(5, device=dev) + (skip + 1) * page
    ds.dflash_store_kv(x, x, slots, *big)
    assert torch.equal(big[0][skip + 1, :5], x) and torch.equal(big[1][skip + 1, :5], x)
    clean()


def test_attention_interleaved_cache(dev):
    """Keys and values interleaved in one tensor: both caches are strided views of it."""
    b = paged.Batch([100, 7], [5, 90], 4, 2, 128, 16, seed=2)
    both = torch.stack([b.key_cache, b.value_cache], dim=1)
    got = ds.dflash_paged_attention(b.query, both[:, 0], both[:, 1], *b.args()[3:])
    for g, w in zip(got, ds.dflash_paged_attention(*b.args())):
        assert torch.equal(g, w)
    clean()


def test_attention_equal_calls_and_streams(dev):
    """Equal calls give equal bits, also on another stream and from a captured graph."""
    b = paged.Batch([5000, 100, 0, 777], [1, 16, 300, 3], 8, 2, 128, 16, seed=12)
    want = ds.dflash_paged_attention(*b.args())
    for _ in range(3):
        for g, w in zip(ds.dflash_paged_attention(*b.args()), want):
            assert torch.equal(g, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(ds.dflash_paged_attention_workspace_bytes(4, b.T, 8, 2, 128),
                     dtype=torch.uint8, device=dev)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ds.dflash_paged_attention(*b.args(), out=out, lse=lse, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.dflash_paged_attention(*b.args(), out=out, lse=lse, workspace=ws)
    b.query.mul_(0.5)
    graph.replay()
    for g, w in zip((out, lse), ds.dflash_paged_attention(*b.args())):
        assert torch.equal(g, w)
    clean()


def test_attention_alone_or_in_a_batch(dev):
    """A request's result in a batch and alone agree within the bounds of each (the split of its
    sums may differ, nothing else does)."""
    b = paged.Batch([3000, 20, 900], [16, 1, 33], 8, 4, 128, 32, seed=13)
    want = paged.attention(b)
    paged.assert_attention(ds.dflash_paged_attention(*b.args()), want)
    t0 = 0
    for r, n in enumerate(b.new.tolist()):
        got = ds.dflash_paged_attention(
            b.query[t0:t0 + n], b.key_cache, b.value_cache, b.block_table[r:r + 1],
            torch.tensor([0, n], dtype=torch.int32, device=dev), b.kv_lens[r:r + 1])
        paged.assert_attention(got, tuple(w[t0:t0 + n] for w in want), f"request {r}")
        t0 += n
    clean()


@pytest.mark.parametrize("seed", range(24))
def test_attention_random(dev, seed):
    """Seeded random shapes, types, windows and lengths."""
    rng = np.random.default_rng(100 + seed)
    dtype, cache = TYPES[rng.integers(4)]
    Hkv = int(rng.integers(1, 5))
    R = int(rng.integers(1, 7))
    ctx = np.exp(rng.uniform(0, 7, R)).astype(int) - 1
    new = np.exp(rng.uniform(0, rng.uniform(0.1, 6), R)).astype(int)
    b = paged.Batch(ctx, new, Hkv * int(rng.integers(1, 10)), Hkv, int(rng.choice([64, 128])),
                    int(rng.choice([8, 16, 32, 64, 128, 256])), dtype, cache,
                    layout=str(rng.choice(["nhd", "hnd"])), seed=seed,
                    spread=float(rng.choice([1.0, 4.0])))
    left = int(rng.choice([-1, -1, 0, 40, 400]))
    check(b, f"seed {seed}", left=left, right=int(rng.choice([0, 0, -1, 9])),
          softcap=float(rng.choice([0.0, 0.0, 20.0])))


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("small", [False, True])
def test_steps_together(dev, small):
    """Three steps as a serving loop runs them (tables, store, attention), the second one's
    tokens partly rejected, against attention over the tokens kept."""
    g = torch.Generator().manual_seed(20)
    R, H, G, D, page, width = 5, 2, 3, 64, 16, 12
    pool = torch.randperm(R * width, generator=g).to(torch.int32).to(dev)
    table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
    dt = E4 if small else BF
    kc = torch.full((R * width, page, H, D), float("nan")).to(dt).to(dev)
    vc = kc.clone()
    ks, vs = (0.05, 0.04) if small else (1.0, 1.0)
    ctx = np.zeros(R, np.int64)
    held = torch.zeros(R, dtype=torch.int32, device=dev)
    at = 0
    kept = [([], []) for _ in range(R)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)               # noqa: E731
    for step, new in enumerate([[40, 3, 17, 1, 64], [16] * 5, [9, 1, 16, 2, 7]]):
        T = sum(new)
        qs, kv, held, pos, slots, needed = ds.dflash_block_tables(
            i32(ctx), i32(new), held, pool[at:].contiguous(), table, page, T)
        at += int(needed)
        qkv = torch.randn((T, H * (G + 2), D), generator=g).to(BF)
        d = qkv.to(dev)
        ds.dflash_store_kv(d[:, H * G:H * (G + 1)], d[:, H * (G + 1):], slots, kc, vc, ks, vs)
        got = ds.dflash_paged_attention(d[:, :H * G], kc, vc, table, qs, kv, k_scale=ks,
                                        v_scale=vs)
        b = paged.Batch.__new__(paged.Batch)
        b.Hq, b.Hkv, b.D, b.dtype, b.T, b.qkv = H * G, H, D, BF, T, qkv
        b.ctx, b.new, b.kv, b.k_scale, b.v_scale = ctx, np.array(new), ctx + new, ks, vs
        b.k, b.v, t0 = [], [], 0
        for r, n in enumerate(new):
            for rows, c, s in ((kept[r][0], H * G, ks), (kept[r][1], H * (G + 1), vs)):
                x = qkv[t0:t0 + n, c:c + H]
                rows.append((x.float() / s).to(E4).float() if small else x)
            b.k.append(torch.cat(kept[r][0]))
            b.v.append(torch.cat(kept[r][1]))
            t0 += n
        paged.assert_attention(got, paged.attention(b), f"step {step}")
        ctx = ctx + new
        if step == 1:                                    # all but 5 tokens of the block rejected
            ctx = ctx - 11
            kept = [tuple([torch.cat(x)[:int(c)]] for x in k) for k, c in zip(kept, ctx)]
    clean()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (10, 2), (16, 1)])
def test_attention_few_rows_on_average(dev, dtype, cache, D, Hq, Hkv):
    """Few rows a request on average, among them requests of many row tiles, of no new tokens and
    of one cached token: all take the build for few rows, whose tiles hold 32 // g tokens."""
    rng = np.random.default_rng(16)
    new = np.where(rng.random(150) < 0.05, rng.integers(5, 60, 150), rng.integers(0, 2, 150))
    assert new.sum() * (Hq // Hkv) <= 32 * len(new) and new.max() * (Hq // Hkv) > 128
    ctx = np.where(rng.random(150) < 0.3, 0, rng.integers(0, 900, 150))
    b = paged.Batch(ctx, new, Hq, Hkv, D, 16, dtype, cache, seed=16)
    want = check(b)
    for _ in range(5):
        for g, w in zip(ds.dflash_paged_attention(*b.args(), **b.scales()), want):
            assert torch.equal(g, w)
    check(b, left=150, right=4, softcap=15.0)
