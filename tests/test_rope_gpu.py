"""The norm and rotation of queries and keys, alone and with the store, against the 64-bit form."""

from __future__ import annotations

import pytest
import torch

import step
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


class Case:
    """Queries, keys and values as slices of a fused projection's output, positions, weights."""

    def __init__(self, dev, T, Hq, Hkv, D, dtype=BF, rotary=None, interleaved=False, norm="qk",
                 weight_dtype=None, far=5000, seed=0, rope_scale=1.0, **freq):
        g = torch.Generator().manual_seed(seed)
        self.T, self.Hq, self.Hkv, self.D, self.dtype = T, Hq, Hkv, D, dtype
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g) * torch.exp(torch.randn((Hq + 2 * Hkv, D), generator=g))
        self.qkv = qkv.to(dtype).to(dev)
        self.query = self.qkv[:, :Hq] if Hq else None
        self.key = self.qkv[:, Hq:Hq + Hkv] if Hkv else None
        self.value = self.qkv[:, Hq + Hkv:]
        self.positions = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).to(dev)
        w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(weight_dtype or dtype).to(dev)   # noqa: E731
        self.q_weight, self.k_weight = (w() if "q" in norm else None), (w() if "k" in norm else None)
        rotary = D if rotary is None else rotary
        self.frequencies = ds.dflash_rope_frequencies(rotary, device=dev, **freq) if rotary else None
        self.how = dict(frequencies=self.frequencies, q_weight=self.q_weight, k_weight=self.k_weight,
                        interleaved=interleaved, rope_scale=rope_scale)
        self.slots = torch.randperm(3 * T + 7, generator=g)[:T].to(dev)

    def want(self, x, weight, eps=1e-6):
        f = [] if self.frequencies is None else self.frequencies.tolist()
        return step.norm_rope(x, weight, eps, step.turns(self.positions.tolist(), f),
                              self.how["interleaved"], self.how["rope_scale"])

    def run(self, **kw):
        return ds.dflash_qk_norm_rope(self.query, self.key, self.positions, **{**self.how, **kw})

    def check(self, got):
        for x, w, y in ((self.query, self.q_weight, got[0]), (self.key, self.k_weight, got[1])):
            if x is None:
                assert y is None
            else:
                assert y.dtype == self.dtype
                step.close_heads(y, *self.want(x, w), self.dtype)
        clean()


SIZES = [(1, 1, 1, 128, 128), (1, 16, 8, 128, 128), (3, 4, 1, 64, 64), (17, 5, 5, 80, 80), (300, 3, 1, 96, 96),
         (9, 2, 2, 8, 8), (33, 2, 1, 16, 16), (5, 3, 2, 72, 72), (40, 4, 2, 256, 256), (129, 7, 1, 24, 24),
         (11, 2, 2, 128, 64), (11, 2, 2, 128, 32), (11, 2, 2, 128, 0), (11, 2, 2, 80, 40), (11, 2, 2, 80, 20),
         (7, 2, 2, 96, 24), (7, 2, 2, 128, 2), (7, 2, 2, 64, 62), (7, 1, 3, 248, 34), (64, 0, 1, 128, 128),
         (64, 1, 0, 128, 128), (513, 0, 1, 16, 16), (5, 130, 1, 64, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,Hq,Hkv,D,rotary", SIZES)
def test_against_64_bits(dev, T, Hq, Hkv, D, rotary, dtype, interleaved):
    c = Case(dev, T, Hq, Hkv, D, dtype, rotary, interleaved, seed=T + D)
    c.check(c.run())


@pytest.mark.parametrize("norm", ["", "q", "k"])
@pytest.mark.parametrize("weight_dtype", [None, torch.float32])
def test_norms_and_weights(dev, norm, weight_dtype):
    c = Case(dev, 21, 3, 2, 64, norm=norm, weight_dtype=weight_dtype, rope_scale=1.25)
    c.check(c.run())


def test_far_positions(dev):
    """Angles stay exact up to the ends of 32 bits; position 0 turns nothing; negative ones turn back."""
    for interleaved in (False, True):
        c = Case(dev, 8, 2, 1, 64, FP, interleaved=interleaved, norm="")
        c.positions = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 0, 1, -1, 999999999, 16777217],
                                   dtype=torch.int32, device=dev)
        got = c.run()
        c.check(got)
        assert torch.equal(got[0][3], c.query[3])


@pytest.mark.parametrize("freq", [dict(factor=8.0), dict(factor=16.0, original_len=4096),
                                  dict(base=500000.0, factor=4.0, original_len=8192, turns_slow=1.0,
                                       turns_fast=4.0),
                                  dict(inv_freq=torch.linspace(1, -0.5, 32))])
def test_scaled_frequencies(dev, freq):
    c = Case(dev, 30, 2, 2, 64, far=200000, rope_scale=1.3, **freq)
    c.check(c.run())


def test_strided_outputs_and_in_place(dev):
    """Outputs into slices of larger tensors, heads apart, and over their inputs."""
    c = Case(dev, 23, 4, 2, 128)
    want = c.run()
    room = torch.full((23, 9, 2, 128), 7.0, dtype=BF, device=dev)
    got = c.run(query_out=room[:, :4, 1], key_out=room[:, 5:7, 0])
    assert got[0].data_ptr() == room[:, :4, 1].data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[:, :, 0][:, :5] == 7).all() and (room[:, 4:, 1] == 7).all() and (room[:, 7:, 0] == 7).all()
    value = c.value.clone()
    c.run(query_out=c.query, key_out=c.key)
    assert torch.equal(c.query, want[0]) and torch.equal(c.key, want[1])
    assert torch.equal(c.value, value)
    clean()


def test_values_that_are_no_numbers(dev):
    """NaN and infinities stay in their own head; zeros stay zeros; values whose squares pass fp32's
    range are normed all the same."""
    c = Case(dev, 6, 3, 1, 128, norm="qk")
    want = c.run()[0]
    c.qkv[1, 0, 5] = float("nan")
    c.qkv[2, 1, 7] = float("inf")
    c.qkv[3, 2] = 0
    got = c.run()[0]
    assert torch.isnan(got[1, 0]).all() and torch.isnan(got[2, 1]).any()
    assert not got[3, 2].any()
    keep = torch.ones((6, 3), dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = keep[3, 2] = False
    assert torch.equal(got[keep.to(dev)], want[keep.to(dev)])
    big = Case(dev, 6, 3, 1, 128)
    big.qkv[4] = (big.qkv[4].float().clamp(-3, 3) * 2.0 ** 125).to(BF)
    big.qkv[5, 0, 3] = torch.finfo(BF).max
    big.check(big.run())


def test_no_tokens(dev):
    c = Case(dev, 4, 2, 1, 64)
    q, k = ds.dflash_qk_norm_rope(c.query[:0], c.key[:0], c.positions[:0], **c.how)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    clean()


# ----------------------------------------------------------------------------- with the store

def caches(dev, pages, page, Hkv, D, dtype, layout="nhd"):
    if layout == "hnd":
        make = lambda: torch.zeros((pages, Hkv, page, D), device=dev).to(dtype).transpose(1, 2)  # noqa: E731
    else:
        make = lambda: torch.zeros((pages, page, Hkv, D), device=dev).to(dtype)                  # noqa: E731
    return make(), make()


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,interleaved", [
    (1, 4, 1, 128, 16, False), (50, 8, 2, 64, 24, False), (33, 3, 3, 80, 16, True), (130, 0, 2, 128, 7, False),
    (700, 1, 1, 16, 32, False), (20, 2, 1, 256, 64, True), (20, 2, 1, 72, 5, False)])
def test_store_is_the_two_calls(dev, T, Hq, Hkv, D, page, interleaved, layout):
    """Into a 16-bit cache: bit for bit the norm and rotation, then the store."""
    for dtype in (BF, FP):
        c = Case(dev, T, Hq, Hkv, D, dtype, interleaved=interleaved, seed=D)
        pages = -(-(3 * T + 7) // page)
        kc, vc = caches(dev, pages, page, Hkv, D, dtype, layout)
        q, gk, gv = ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc, **c.how)
        assert gk is kc and gv is vc
        wq, wk = c.run()
        k2, v2 = caches(dev, pages, page, Hkv, D, dtype, layout)
        ds.dflash_store_kv(wk, c.value, c.slots, k2, v2)
        assert torch.equal(kc, k2) and torch.equal(vc, v2)
        assert q is None if Hq == 0 else torch.equal(q, wq)
    clean()


@pytest.mark.parametrize("k_scale,v_scale", [(0.0625, 0.03125), (0.07, 0.3)])
@pytest.mark.parametrize("D,interleaved", [(128, False), (64, True), (80, False), (96, False)])
def test_store_e4m3(dev, D, interleaved, k_scale, v_scale):
    """Keys are rounded once, values as dflash_store_kv rounds them."""
    rotary = D // 4 if D == 96 else D
    c = Case(dev, 77, 4, 2, D, rotary=rotary, interleaved=interleaved)
    kc, vc = caches(dev, 17, 16, 2, D, E4)
    q, _, _ = ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc,
                                           k_scale=k_scale, v_scale=v_scale, **c.how)
    step.close_heads(q, *c.want(c.query, c.q_weight), BF)
    k2, v2 = caches(dev, 17, 16, 2, D, E4)
    ds.dflash_store_kv(c.key, c.value, c.slots, k2, v2, k_scale=k_scale, v_scale=v_scale)
    assert torch.equal(vc.view(torch.uint8), v2.view(torch.uint8))
    stored = kc.float().flatten(0, 1)[c.slots]
    step.close_e4m3(stored, *c.want(c.key, c.k_weight), torch.tensor(k_scale).item())
    empty = torch.ones(17 * 16, dtype=torch.bool, device=dev)
    empty[c.slots] = False
    assert not kc.float().flatten(0, 1)[empty].any()
    clean()


def test_slots_that_store_nothing(dev):
    """Padded tokens (slot -1) and slots outside the cache; their queries are written all the same."""
    c = Case(dev, 40, 2, 2, 64)
    want = c.run()[0]
    kc, vc = caches(dev, 9, 16, 2, 64, BF)
    c.slots = torch.arange(40, device=dev)
    c.slots[::3] = -1
    q, _, _ = ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc, **c.how)
    assert torch.equal(q, want)
    at = (c.slots >= 0).nonzero()[:, 0]
    rows = vc.flatten(0, 1)
    assert torch.equal(rows[at], c.value[at]) and not rows[40:].any() and not rows[0:40:3].any()
    clean()
    c.slots[1] = 9 * 16
    c.slots[2] = 2 ** 40
    ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc, **c.how)
    assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_ID


def test_values_are_copied_bit_by_bit(dev):
    c = Case(dev, 3, 1, 1, 64)
    bits = torch.arange(3 * 64, dtype=torch.int32).mul(341).to(torch.int16).view(3, 1, 64).to(dev)
    kc, vc = caches(dev, 2, 16, 1, 64, BF)
    c.slots = torch.tensor([3, 20, 31], device=dev)
    ds.dflash_qk_norm_rope_store(None, c.key, bits.view(BF), c.positions, c.slots, kc, vc, **c.how)
    assert torch.equal(vc.flatten(0, 1)[c.slots].view(torch.int16), bits)
    clean()


def test_cache_past_2_to_the_31_elements(dev):
    """Slots at the far end of a cache of more than 2^31 elements."""
    if torch.cuda.mem_get_info(dev)[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB of device memory")
    kc = torch.zeros((2 ** 31 // (64 * 128) + 3, 64, 2, 64), dtype=BF, device=dev)
    vc = torch.zeros_like(kc)
    c = Case(dev, 5, 2, 2, 64)
    last = kc.shape[0] * 64 - 1
    c.slots = torch.tensor([last, 0, last // 2, last - 64, 2 ** 24 + 3])
    assert int(c.slots.max()) == last and len(set(c.slots.tolist())) == 5
    c.slots = c.slots.to(dev)
    ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc, **c.how)
    assert torch.equal(vc.flatten(0, 1)[c.slots], c.value)
    assert torch.equal(kc.flatten(0, 1)[c.slots], c.run()[1])
    clean()


def test_in_a_graph(dev):
    c = Case(dev, 40, 4, 2, 128)
    kc, vc = caches(dev, 9, 16, 2, 128, BF)
    out = torch.empty((40, 4, 128), dtype=BF, device=dev)
    call = lambda: ds.dflash_qk_norm_rope_store(c.query, c.key, c.value, c.positions, c.slots, kc, vc,  # noqa: E731
                                                query_out=out, **c.how)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.qkv.copy_(torch.randn_like(c.qkv))
    c.positions.add_(5)
    kc.zero_()
    graph.replay()
    wq, wk = c.run()
    torch.cuda.synchronize()
    assert torch.equal(out, wq) and torch.equal(kc.flatten(0, 1)[c.slots], wk)
    clean()
