"""The paged cache operators without a GPU: refusals of bad arguments before any CUDA call, and
the plain forms that the GPU tests compare with, checked on worked cases."""

import ctypes
import math

import numpy as np
import pytest
import torch

import paged
import draft_candidate_selector_gb300 as ds
from draft_candidate_selector_gb300 import _native

P = ctypes.c_void_p
A, MIS, NULL = P(4096), P(4100), P(None)
BAD, UNS, WS = (_native.DFLASH_INVALID_ARGUMENT, _native.DFLASH_UNSUPPORTED,
                _native.DFLASH_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def cache(**kw):
    d = dict(key=4096, value=4096, page_stride=16 * 128, token_stride=128, head_stride=64,
             num_pages=8, page_size=16, kv_heads=2, head_dim=64, dtype=_native.BF16, k_scale=1.0,
             v_scale=1.0)
    d.update(kw)
    return _native.KvCache(**d)


BAD_CACHES = [
    (dict(key=None), BAD), (dict(value=4100), BAD), (dict(num_pages=0), BAD),
    (dict(page_size=0), BAD), (dict(kv_heads=0), BAD), (dict(head_dim=0), BAD),
    (dict(head_dim=60), UNS), (dict(head_dim=264), UNS), (dict(token_stride=-128), BAD),
    (dict(token_stride=130), UNS), (dict(page_stride=2052), UNS), (dict(head_stride=4), UNS),
    (dict(dtype=7), BAD), (dict(dtype=_native.FP16), BAD), (dict(k_scale=0.5), BAD),
    (dict(dtype=_native.E4M3, k_scale=0.0), BAD),
    (dict(dtype=_native.E4M3, v_scale=math.inf), BAD),
    (dict(dtype=_native.E4M3, v_scale=math.nan), BAD),
    (dict(dtype=_native.E4M3, head_dim=72), UNS),
    (dict(dtype=_native.E4M3, head_stride=8), UNS),
]


def store(lib, c, key=A, value=A, dtype=_native.BF16, slots=A, T=5, strides=(128, 64, 128, 64)):
    return lib.dflash_store_kv(key, value, dtype, slots, T, *strides, ctypes.byref(c), None)


def attend(lib, c, query=A, dtype=_native.BF16, T=5, Hq=4, strides=(256, 64), table=A, R=2,
           width=4, start=A, kv=A, scale=1.0, left=-1, right=0, cap=0.0, out=A, lse=A, ws=A,
           wsb=1 << 40):
    return lib.dflash_paged_attention(query, dtype, T, Hq, *strides, ctypes.byref(c), table, R,
                                      width, start, kv, scale, left, right, cap, out, lse, ws,
                                      wsb, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, status):
    assert store(lib, cache(**change)) == status
    assert attend(lib, cache(**change)) == status
    assert lib.dflash_last_error()


def test_store_refusals(lib):
    assert store(lib, cache(), key=NULL) == BAD
    assert store(lib, cache(), value=MIS) == BAD
    assert store(lib, cache(), slots=MIS) == BAD
    assert store(lib, cache(), T=-1) == BAD
    assert store(lib, cache(), dtype=_native.E4M3) == BAD
    for i in range(4):
        s = [128, 64, 128, 64]
        s[i] = 12
        assert store(lib, cache(), strides=s) == UNS
        s[i] = -8
        assert store(lib, cache(), strides=s) == BAD
    assert lib.dflash_store_kv(A, A, 0, A, 5, 128, 64, 128, 64, None, None) == BAD
    assert store(lib, cache(), key=NULL, T=0) == _native.DFLASH_OK


def test_attention_refusals(lib):
    for name in ("query", "table", "start", "kv", "out", "ws"):
        assert attend(lib, cache(), **{name: NULL}) == BAD
    for name in ("query", "out", "ws"):
        assert attend(lib, cache(), **{name: MIS}) == BAD
    assert attend(lib, cache(), lse=P(4098)) == BAD
    assert attend(lib, cache(), T=-1) == BAD
    assert attend(lib, cache(), R=0) == BAD
    assert attend(lib, cache(), width=0) == BAD
    assert attend(lib, cache(), Hq=0) == BAD
    assert attend(lib, cache(), Hq=3) == BAD
    assert attend(lib, cache(), dtype=2) == BAD
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert attend(lib, cache(), scale=scale) == BAD
    for cap in (-1.0, math.nan, math.inf):
        assert attend(lib, cache(), cap=cap) == BAD
    assert attend(lib, cache(), left=-2) == BAD
    assert attend(lib, cache(), right=-2) == BAD
    assert attend(lib, cache(), strides=(12, 64)) == UNS
    assert attend(lib, cache(), strides=(256, -64)) == BAD
    assert attend(lib, cache(), T=1 << 30) == BAD
    assert attend(lib, cache(), T=0, query=NULL) == _native.DFLASH_OK


def test_block_table_refusals(lib):
    good = dict(ctx=A, new=A, held=P(8192), free=A, R=2, n=3, page=16, width=4, T=5, table=A,
                start=A, kv=P(8192), held_out=A, pos=A, slots=A, needed=A)

    def call(**kw):
        return lib.dflash_block_tables(*{**good, **kw}.values(), None)

    for name in ("ctx", "new", "held", "free", "table", "start", "kv", "held_out", "pos", "slots",
                 "needed"):
        assert call(**{name: NULL}) == BAD
        assert call(**{name: P(4098)}) == BAD
    assert call(slots=MIS) == BAD
    assert call(held_out=P(8192)) == BAD
    assert call(kv=A) == BAD
    for name in ("R", "page", "width"):
        assert call(**{name: 0}) == BAD
    assert call(T=-1) == BAD
    assert call(n=-1) == BAD
    assert call(R=16385) == UNS


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks behaviour without a GPU")
def test_no_device_is_reported(lib):
    none = _native.DFLASH_NO_DEVICE
    assert store(lib, cache()) == none
    assert attend(lib, cache()) == none
    assert lib.dflash_paged_attention_workspace_bytes(2, 5, 4, 2, 64) == 0
    assert lib.dflash_block_tables(A, A, P(8192), A, 2, 3, 16, 4, 5, A, A, P(8192), A, A, A, A,
                                   None) == none


def test_python_refusals():
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((3,), dtype=torch.int64)
    with pytest.raises(TypeError):
        ds.dflash_store_kv(None, x, i, c, c)
    with pytest.raises(ValueError, match="CUDA"):
        ds.dflash_store_kv(x, x, i, c, c)
    with pytest.raises(ValueError, match="CUDA"):
        ds.dflash_paged_attention(x, c, c, i, i, i)
    with pytest.raises(ValueError):
        ds.dflash_block_tables(i, i, i, i, c, 16, 3)
    with pytest.raises(ValueError):
        ds.dflash_block_tables(i, i, i, i, torch.zeros((3, 4), dtype=torch.int32), 16, 3)


def test_plain_tables_worked():
    """Two requests on pages of 4: 3 cached tokens in one page plus 6 new need two more pages; 4
    cached in one page plus 0 new need none; then one that the list is too short for."""
    table = np.array([[5, -1, -1], [6, -1, -1], [-1, -1, -1]])
    t, start, kv, held, pos, slots, needed, refused = paged.tables(
        [3, 4, 0], [6, 0, 1], [1, 1, 0], [9, 2], table, 4, 8)
    assert t.tolist() == [[5, 9, 2], [6, -1, -1], [-1, -1, -1]]
    assert start.tolist() == [0, 6, 6, 7] and kv.tolist() == [9, 4, 0]
    assert held.tolist() == [3, 1, 0] and needed == 3 and refused.tolist() == [0, 0, 1]
    assert pos.tolist() == [3, 4, 5, 6, 7, 8, 0, 0]
    assert slots.tolist() == [23, 36, 37, 38, 39, 8, -1, -1]


def test_plain_attention_against_closed_forms():
    """One visible key returns its value; equal keys return the mean of the visible values; an
    empty row is zero; the log-sum-exp of n equal scores s is s + log n."""
    b = paged.Batch([0, 3], [4, 2], 2, 1, 64, 8, device="cpu", dtype=torch.float16)
    out, lse, _, _ = paged.attention(b, left=0, right=0)
    assert torch.allclose(out[:4, 0], b.v[0][:, 0].double())
    b.k[1][:] = b.k[1][:1]
    out, lse, _, _ = paged.attention(b)
    v = b.v[1][:, 0].double()
    assert torch.allclose(out[4, 1], v[:4].mean(0)) and torch.allclose(out[5, 1], v.mean(0))
    s = float(b.qkv[5, 1].double() @ b.k[1][0, 0].double()) / 8
    assert abs(float(lse[5, 1]) - s - math.log(5)) < 1e-12
    b.kv[0] = 0
    assert not paged.attention(b)[0][:4].any() and torch.isinf(paged.attention(b)[1][:4]).all()
