"""The sampled step's operators without a GPU: frequencies, refusals before any CUDA call, and the plain
forms that the GPU tests compare with, checked on worked cases."""

from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import step
from test_paged_calls import placed
from test_paged_host import A, BAD, MIS, NULL, P, UNS, WS, cache
import draft_candidate_selector_gb300 as ds
from draft_candidate_selector_gb300 import _native

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    return _native.load()


# ----------------------------------------------------------------------------- frequencies

TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021")


def near(got, radians):
    """A frequency is off by three roundings to 53 bits and half of 2^-64."""
    got = [Fraction(int(g) % 2 ** 64, 2 ** 64) for g in got]
    for g, f in zip(got, radians):
        want = Fraction(float(f)) / TWO_PI % 1
        off = min(abs(g - want), 1 - abs(g - want))
        assert off <= abs(Fraction(float(f))) / TWO_PI * Fraction(1, 2 ** 50) + Fraction(1, 2 ** 63)


def test_frequencies():
    f = 10000.0 ** (-2 * np.arange(64) / 128)
    near(ds.dflash_rope_frequencies(128, device="cpu").tolist(), f)
    near(ds.dflash_rope_frequencies(128, factor=8.0, device="cpu").tolist(), f / 8)
    turns = 4096 * f / (2 * math.pi)
    got = ds.dflash_rope_frequencies(128, factor=4.0, original_len=4096, device="cpu").tolist()
    keep = np.clip((turns - 1) / 31, 0, 1)
    assert keep[0] == 1 and keep[-1] == 0 and ((keep > 0) & (keep < 1)).any()
    near(got, f / 4 * (1 - keep) + f * keep)
    own = torch.tensor([0.0, 1.0, -1.0, 100.0, 2 * math.pi, 1e-9])
    near(ds.dflash_rope_frequencies(12, inv_freq=own, device="cpu").tolist(), own.double().tolist())
    assert ds.dflash_rope_frequencies(0, device="cpu").shape == (0,)


def test_frequency_refusals():
    for kw in (dict(rotary_dim=-2), dict(rotary_dim=7), dict(base=0.0), dict(base=math.inf), dict(factor=0.0),
               dict(factor=math.nan), dict(original_len=-1.0), dict(original_len=math.inf),
               dict(original_len=10, turns_slow=2.0, turns_fast=2.0),
               dict(inv_freq=torch.tensor([1.0, math.nan])), dict(inv_freq=torch.ones(3))):
        with pytest.raises(ValueError):
            ds.dflash_rope_frequencies(**{"rotary_dim": 4, "device": "cpu", **kw})


# ----------------------------------------------------------------------------- refusals

def how(**kw):
    d = dict(q_weight=4096, k_weight=4096, weight_dtype=_native.BF16, eps=1e-6, frequencies=4096,
             rotary_dim=64, interleaved=0, rope_scale=1.0)
    d.update(kw)
    return _native.NormRope(**d)


def rope(lib, h=None, query=A, key=A, dtype=_native.BF16, positions=A, T=5, Hq=4, Hkv=2, D=64,
         strides=(256, 64, 128, 64), qo=A, ko=A, out=(256, 64, 128, 64)):
    return lib.dflash_qk_norm_rope(query, key, dtype, positions, T, Hq, Hkv, D, *strides,
                                   ctypes.byref(h or how()), qo, ko, *out, None)


def rope_store(lib, h=None, c=None, query=A, key=A, value=A, dtype=_native.BF16, positions=A, slots=A, T=5,
               Hq=4, strides=(256, 64, 128, 64, 128, 64), qo=A, out=(256, 64)):
    return lib.dflash_qk_norm_rope_store(query, key, value, dtype, positions, slots, T, Hq, *strides,
                                         ctypes.byref(h or how()), ctypes.byref(c or cache()), qo, *out, None)


@pytest.mark.parametrize("change,status", [
    (dict(weight_dtype=_native.FP16), BAD), (dict(weight_dtype=_native.E4M3), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD), (dict(frequencies=None), BAD),
    (dict(frequencies=4100), BAD), (dict(rotary_dim=-2), BAD), (dict(rotary_dim=63), BAD),
    (dict(rotary_dim=66), BAD), (dict(rope_scale=math.inf), BAD), (dict(rope_scale=math.nan), BAD),
    (dict(q_weight=4097), BAD), (dict(k_weight=4098, weight_dtype=_native.FP32), BAD)])
def test_norm_rope_parameters(lib, change, status):
    assert rope(lib, how(**change)) == status
    assert rope_store(lib, how(**change)) == status
    assert lib.dflash_last_error()


def test_norm_rope_refusals(lib):
    for name in ("query", "key", "qo", "ko"):
        assert rope(lib, **{name: NULL}) == BAD
        assert rope(lib, **{name: MIS}) == BAD
    assert rope(lib, positions=NULL) == BAD and rope(lib, positions=P(4098)) == BAD
    assert rope(lib, T=-1) == BAD and rope(lib, Hq=-1) == BAD and rope(lib, Hkv=-1) == BAD
    assert rope(lib, Hq=0, Hkv=0) == BAD
    assert rope(lib, D=0) == BAD and rope(lib, D=60) == UNS and rope(lib, D=264) == UNS
    assert rope(lib, dtype=_native.E4M3) == BAD and rope(lib, dtype=_native.FP32) == BAD
    assert rope(lib, T=2 ** 30) == BAD and rope(lib, T=1, Hq=2 ** 31 - 1) == BAD
    for i in range(4):
        for at in ("strides", "out"):
            s = [256, 64, 128, 64]
            s[i] = 12
            assert rope(lib, **{at: s}) == UNS
            s[i] = -8
            assert rope(lib, **{at: s}) == BAD
    assert rope(lib, T=0, query=NULL, key=NULL, qo=NULL) == _native.DFLASH_OK
    assert lib.dflash_qk_norm_rope(A, A, 0, A, 5, 4, 2, 64, 256, 64, 128, 64, None, A, A, 256, 64, 128, 64,
                                   None) == BAD


def test_norm_rope_store_refusals(lib):
    for name in ("query", "key", "value", "qo"):
        assert rope_store(lib, **{name: NULL}) == BAD
        assert rope_store(lib, **{name: MIS}) == BAD
    assert rope_store(lib, slots=NULL) == BAD and rope_store(lib, slots=MIS) == BAD
    assert rope_store(lib, T=-1) == BAD and rope_store(lib, Hq=-1) == BAD
    assert rope_store(lib, c=cache(head_dim=264)) == UNS and rope_store(lib, c=cache(dtype=_native.FP16)) == BAD
    for i in range(6):
        s = [256, 64, 128, 64, 128, 64]
        s[i] = 12
        assert rope_store(lib, strides=s) == UNS
    assert rope_store(lib, T=0, key=NULL, slots=NULL) == _native.DFLASH_OK


def path(lib, edges=A, ids=A, u=A, temps=NULL, t=1.0, R=2, S=3, K=4, path=A, tokens=A, probs=A):
    return lib.dflash_sample_path(edges, ids, u, temps, t, R, S, K, path, tokens, probs, None)


def test_sample_path_refusals(lib):
    for name in ("edges", "ids", "u", "path", "tokens", "probs"):
        assert path(lib, **{name: NULL}) == BAD and path(lib, **{name: P(4098)}) == BAD
    assert path(lib, temps=P(4098)) == BAD
    for name in ("R", "S", "K"):
        assert path(lib, **{name: 0}) == BAD
    assert path(lib, K=33) == UNS and path(lib, S=257) == UNS
    for t in (-0.5, math.nan, math.inf):
        assert path(lib, t=t) == BAD


def verify(lib, logits=A, dtype=_native.BF16, T=8, V=100, stride=100, start=A, drafts=A, R=2, S=3, ids=A,
           probs=A, K=4, accept=A, sample=A, temps=NULL, t=1.0, tokens=A, counts=A, logprobs=A, ws=A,
           wsb=1 << 40):
    return lib.dflash_verify_drafts(logits, dtype, T, V, stride, start, drafts, R, S, ids, probs, K, accept,
                                    sample, temps, t, tokens, counts, logprobs, ws, wsb, None)


def test_verify_refusals(lib):
    for name in ("logits", "start", "drafts", "accept", "sample", "tokens", "counts", "ws"):
        assert verify(lib, **{name: NULL}) == BAD
        assert verify(lib, **{name: P(4097)}) == BAD
    assert verify(lib, logits=P(4098), dtype=_native.FP32) == BAD
    assert verify(lib, ids=NULL) == BAD and verify(lib, probs=NULL) == BAD
    assert verify(lib, ids=P(4098)) == BAD and verify(lib, probs=P(4098)) == BAD
    assert verify(lib, logprobs=P(4098)) == BAD and verify(lib, ws=MIS) == BAD
    assert verify(lib, dtype=_native.E4M3) == BAD and verify(lib, dtype=9) == BAD
    for name in ("V", "R"):
        assert verify(lib, **{name: 0}) == BAD
    assert verify(lib, T=-1) == BAD and verify(lib, S=-1) == BAD and verify(lib, S=256) == UNS
    assert verify(lib, V=2 ** 20 + 1, stride=2 ** 20 + 1) == UNS
    assert verify(lib, stride=99) == BAD and verify(lib, K=0) == BAD and verify(lib, K=33) == UNS
    for t in (-0.5, math.nan, math.inf):
        assert verify(lib, t=t) == BAD
    need = lib.dflash_verify_drafts_workspace_bytes(2, 8, 100)
    assert need > 0 and verify(lib, wsb=need - 1) == WS
    for bad in ((0, 8, 100), (2, -1, 100), (2, 8, 0)):
        assert lib.dflash_verify_drafts_workspace_bytes(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks behaviour without a GPU")
def test_no_device_is_reported(lib):
    none = _native.DFLASH_NO_DEVICE
    assert rope(lib) == none and rope_store(lib) == none and path(lib) == none and verify(lib) == none
    assert rope(lib, how(rotary_dim=0, frequencies=None), positions=NULL) == none
    assert verify(lib, S=0, drafts=NULL, accept=NULL, ids=NULL, probs=NULL) == none


# ----------------------------------------------------------------------------- Python calls

def rope_arguments():
    return dict(query=placed((7, 4, 64), BF), key=placed((7, 2, 64), BF), positions=placed((7,), I32),
                frequencies=placed((32,), torch.int64), q_weight=placed((64,), BF), k_weight=placed((64,), BF),
                query_out=placed((7, 4, 64), BF), key_out=placed((7, 2, 64), BF))


def store_arguments():
    a = rope_arguments()
    del a["key_out"]
    first = dict(key=a.pop("key"), query=a.pop("query"), value=placed((7, 2, 64), BF),
                 slots=placed((7,), torch.int64), key_cache=placed((4, 16, 2, 64), BF),
                 value_cache=placed((4, 16, 2, 64), BF))
    return {**first, **a}


def path_arguments():
    return dict(edges=placed((3, 5, 4, 4), F32), cand_ids=placed((3, 5, 4), I32), uniforms=placed((3, 5), F32),
                temperature=placed((3,), F32), path=placed((3, 5), I32), tokens=placed((3, 5), I32),
                probs=placed((3, 5, 4), F32))


def verify_arguments():
    return dict(logits=placed((12, 50), BF), query_start=placed((4,), I32), draft_tokens=placed((3, 5), I32),
                accept_uniforms=placed((3, 5), F32), sample_uniforms=placed((3,), F32),
                cand_ids=placed((3, 5, 4), I32), draft_probs=placed((3, 5, 4), F32),
                temperature=placed((3,), F32), tokens=placed((3, 6), I32), counts=placed((3,), I32),
                logprobs=placed((3, 6), F32), workspace=placed((1 << 20,), torch.uint8))


CALLS = [(ds.dflash_qk_norm_rope, rope_arguments), (ds.dflash_qk_norm_rope_store, store_arguments),
         (ds.dflash_sample_path, path_arguments), (ds.dflash_verify_drafts, verify_arguments)]


@pytest.mark.parametrize("call,make", CALLS)
def test_wrong_tensors(call, make, monkeypatch):
    """Every tensor on another device than the first, in host memory, of another type or another shape is
    refused before anything is launched."""
    launched = []
    monkeypatch.setattr(ds, "_launch", lambda fn, *a: launched.append(fn))
    call(**make())
    assert len(launched) == 1
    tensors = [n for n, t in make().items()]
    for name in tensors:
        args = make()
        if name != tensors[0]:
            args[name].at = 1
            with pytest.raises(ValueError, match=name):
                call(**args)
        args[name] = args[name].as_subclass(torch.Tensor)
        with pytest.raises(ValueError):
            call(**args)
        if name == "workspace":
            continue
        for wrong in (placed(tuple(make()[name].shape), torch.float64),
                      placed((2,) + tuple(make()[name].shape), make()[name].dtype)):
            args = make()
            args[name] = wrong
            with pytest.raises(ValueError):
                call(**args)
        shape = tuple(make()[name].shape)
        if name not in ("logits", "key_cache", "value_cache", "query", "frequencies"):
            args = make()
            args[name] = placed(shape[:-1] + (shape[-1] + 8,), make()[name].dtype)
            with pytest.raises(ValueError):
                call(**args)
    assert len(launched) == 1


def test_python_refusals(monkeypatch):
    monkeypatch.setattr(ds, "_launch", lambda fn, *a: pytest.fail("launched"))
    with pytest.raises(ValueError, match="both"):
        ds.dflash_qk_norm_rope(None, None, None)
    a = verify_arguments()
    for name in ("cand_ids", "draft_probs"):
        with pytest.raises(ValueError, match="together"):
            ds.dflash_verify_drafts(**{**a, name: None})
    with pytest.raises(ValueError, match="V contiguous"):
        ds.dflash_verify_drafts(**{**a, "logits": placed((12, 100), BF)[:, ::2]})
    with pytest.raises(TypeError, match="logits"):
        ds.dflash_verify_drafts(**{**a, "logits": None})
    with pytest.raises(ValueError, match="strided|contiguous"):
        ds.dflash_sample_path(**{**path_arguments(), "uniforms": placed((3, 10), F32)[:, ::2]})


# ----------------------------------------------------------------------------- the plain forms

def test_plain_rotation_worked():
    """A quarter turn takes (a, b) to (-b, a); the norm of equal values is the weight."""
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0]]])
    quarter = torch.full((1, 2), 0.25, dtype=torch.float64)
    y, _ = step.norm_rope(x, None, 0.0, quarter, False, 1.0)
    assert torch.allclose(y, torch.tensor([[[-3.0, -4.0, 1.0, 2.0]]]).double())
    y, _ = step.norm_rope(x, None, 0.0, quarter[:, :1], True, 2.0)
    assert torch.allclose(y, torch.tensor([[[-4.0, 2.0, 3.0, 4.0]]]).double())
    y, _ = step.norm_rope(torch.full((1, 1, 4), -7.0), torch.tensor([1.0, 2.0, 3.0, 4.0]), 0.0,
                          torch.zeros((1, 0)), False, 1.0)
    assert torch.allclose(y, -torch.tensor([[[1.0, 2.0, 3.0, 4.0]]]).double())
    assert step.turns([3, -1], [2 ** 62, -1])[0, 0] == -0.25


def test_plain_path_worked():
    """Weights 1, 2, 1: quarters of the interval; a border belongs to the candidate behind it."""
    row = torch.log(torch.tensor([1.0, 2.0, 1.0], dtype=torch.float64))
    e = row.expand(1, 1, 3, 3)
    for u, c in ((0.0, 0), (0.2, 0), (0.25, 1), (0.5, 1), (0.74, 1), (0.76, 2), (0.99, 2)):
        path, probs = step.sample_path(e, torch.tensor([[u]]), [1.0])
        if u != 0.25:
            assert path[0, 0] == c
        assert np.allclose(probs[0, 0], [0.25, 0.5, 0.25])
    flat = torch.zeros((1, 2, 4, 4))
    assert step.sample_path(flat, torch.tensor([[0.25, 0.75]]), [1.0])[0].tolist() == [[1, 3]]
    assert step.sample_path(flat + torch.arange(4.0), torch.tensor([[0.1, 0.1]]), [0.0])[0].tolist() == [[3, 3]]


def test_plain_verify_keeps_the_target():
    """Over a fine grid of both uniforms, the first token's frequencies are the target's."""
    logits = torch.log(torch.tensor([[0.1, 0.2, 0.7], [0.3, 0.3, 0.4]], dtype=torch.float64))
    q = torch.tensor([0.6, 0.4])
    n, seen = 40, np.zeros(3)
    for x, mass in ((0, 0.6), (1, 0.4)):
        for i in range(n):
            for j in range(n):
                tokens, counts, _ = step.verify(
                    logits, torch.tensor([0, 2]), torch.tensor([[x]]), torch.tensor([[(i + 0.5) / n]]),
                    torch.tensor([(j + 0.5) / n]), torch.tensor([[[0, 1]]]), q[None, None], [1.0])
                seen[tokens[0, 0]] += mass / n / n
                assert counts[0] == (2 if tokens[0, 1] >= 0 else 1)
    assert np.abs(seen - [0.1, 0.2, 0.7]).max() < 2.0 / n
