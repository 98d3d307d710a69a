"""Calls of the paged operators as users make them: workspaces, caller-given outputs, layouts with
dimensions of one element, tensors of several devices."""

from __future__ import annotations

import pytest
import torch

import paged
import draft_candidate_selector_gb300 as ds

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    ds.dflash_device_status(clear=True)
    return d


@pytest.mark.gpu
def test_no_workspace_where_none_is_used(dev):
    """Head sizes of the CUDA-core kernel, which writes its outputs at once."""
    for D in (8, 80, 96, 192, 256):
        assert 0 < ds.dflash_paged_attention_workspace_bytes(3, 9, 8, 2, D) <= 256
    assert 0 < ds.dflash_paged_attention_workspace_bytes(3, 9, 130, 1, 128) <= 256
    b = paged.Batch([30, 3000], [5, 1], 4, 2, 256, 16, seed=2)
    got = ds.dflash_paged_attention(*b.args(), workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    paged.assert_attention(got, paged.attention(b))
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.gpu
def test_strides_of_one_element(dev):
    """A dimension of one element has no stride that matters: one new token, one key head, one page."""
    b = paged.Batch([5], [1], 2, 1, 64, 16, seed=1, spare_pages=0)
    want = ds.dflash_paged_attention(*b.args())
    q = b.query.as_strided(b.query.shape, (3, b.query.stride(1), 1), b.query.storage_offset())
    s = b.key_cache.stride()
    kc = b.key_cache.as_strided(b.key_cache.shape, (1, s[1], 7, 1))
    vc = b.value_cache.as_strided(b.value_cache.shape, (5, s[1], 64, 1))
    got = ds.dflash_paged_attention(q, kc, vc, *b.args()[3:])
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    x = torch.randn((1, 1, 64), device=dev).to(BF)
    slot = torch.tensor([9], device=dev)
    ds.dflash_store_kv(x.as_strided(x.shape, (3, 5, 1)), x.as_strided(x.shape, (1, 1, 1)), slot, kc, vc)
    assert torch.equal(b.key_cache[0, 9], x[0]) and torch.equal(b.value_cache[0, 9], x[0])
    assert ds.dflash_device_status(clear=True) == 0


class Placed(torch.Tensor):
    """A CPU tensor that says it is on CUDA device `at`: for checks that come before any CUDA call."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at


def placed(shape, dtype, at=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Placed)
    t.at = at
    return t


def table_arguments():
    i = torch.int32
    return dict(context_lens=placed((3,), i), new_lens=placed((3,), i), held_pages=placed((3,), i),
                free_pages=placed((5,), i), block_table=placed((3, 4), i), page_size=16, T=7,
                query_start=placed((4,), i), kv_lens=placed((3,), i), held_out=placed((3,), i),
                positions=placed((7,), i), slots=placed((7,), torch.int64),
                pages_needed=placed((1,), i))


def store_arguments():
    return dict(key=placed((7, 2, 64), BF), value=placed((7, 2, 64), BF),
                slots=placed((7,), torch.int64), key_cache=placed((4, 16, 2, 64), BF),
                value_cache=placed((4, 16, 2, 64), BF))


def attention_arguments():
    return dict(query=placed((7, 4, 64), BF), key_cache=placed((4, 16, 2, 64), BF),
                value_cache=placed((4, 16, 2, 64), BF), block_table=placed((3, 4), torch.int32),
                query_start=placed((4,), torch.int32), kv_lens=placed((3,), torch.int32),
                out=placed((7, 4, 64), BF), lse=placed((7, 4), torch.float32),
                workspace=placed((64,), torch.uint8))


CALLS = [(ds.dflash_block_tables, table_arguments), (ds.dflash_store_kv, store_arguments),
         (ds.dflash_paged_attention, attention_arguments)]


@pytest.mark.parametrize("call,make", CALLS)
def test_tensors_of_several_devices(call, make, monkeypatch):
    """Every tensor on another device than the first is refused before anything is launched, and so
    is a tensor in host memory."""
    launched = []
    monkeypatch.setattr(ds, "_launch", lambda fn, *a: launched.append(fn))
    call(**make())
    assert len(launched) == 1
    tensors = [n for n, t in make().items() if isinstance(t, torch.Tensor)]
    for name in tensors[1:]:
        args = make()
        args[name].at = 1
        with pytest.raises(ValueError, match=name):
            call(**args)
        args[name] = args[name].as_subclass(torch.Tensor)
        with pytest.raises(ValueError, match=name):
            call(**args)
    args = make()
    args[tensors[0]] = args[tensors[0]].as_subclass(torch.Tensor)
    with pytest.raises(ValueError, match="CUDA"):
        call(**args)
    assert len(launched) == 1


@pytest.mark.gpu
def test_workspaces_are_checked(dev):
    b = paged.Batch([100, 3000], [5, 1], 4, 2, 128, 16, seed=2)
    want = ds.dflash_paged_attention(*b.args())
    need = ds.dflash_paged_attention_workspace_bytes(2, b.T, 4, 2, 128)
    u8 = dict(dtype=torch.uint8, device=dev)
    for ws in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, **u8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            ds.dflash_paged_attention(*b.args(), workspace=ws)
    with pytest.raises(TypeError, match="workspace"):
        ds.dflash_paged_attention(*b.args(), workspace=need)
    with pytest.raises(ValueError, match="needed"):       # the library's own answer
        ds.dflash_paged_attention(*b.args(), workspace=torch.empty(need - 1, **u8))
    got = ds.dflash_paged_attention(*b.args(), workspace=torch.empty(-(-need // 4), device=dev))
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.gpu
def test_workspaces_of_the_selector_are_checked(dev):
    logits = torch.randn((2, 3, 70000), device=dev)
    want = ds.dflash_topk_candidates(logits, 8)
    need = ds.dflash_topk_workspace_bytes(2, 3, 70000, 8)
    with pytest.raises(ValueError, match="workspace"):
        ds.dflash_topk_candidates(logits, 8, workspace=torch.empty(need, dtype=torch.uint8))
    got = ds.dflash_topk_candidates(logits, 8, workspace=torch.empty(-(-need // 4), device=dev))
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [("query_start",), ("positions", "slots"), ("slots",),
                                   ("query_start", "kv_lens", "held_out", "positions", "slots",
                                    "pages_needed")])
def test_tables_into_given_outputs(dev, given):
    """Some or all outputs the caller's own: the same values, in the caller's tensors."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)                  # noqa: E731
    args = lambda: (i32(30, 5, 64), i32(40, 9, 1), i32(2, 1, 4), i32(*range(100, 140)),  # noqa: E731
                    torch.arange(30, dtype=torch.int32, device=dev).reshape(3, 10), 16, 55)
    names = ("query_start", "kv_lens", "held_out", "positions", "slots", "pages_needed")
    want = dict(zip(names, ds.dflash_block_tables(*args())))
    own = {n: torch.full_like(want[n], -7) for n in given}
    got = dict(zip(names, ds.dflash_block_tables(*args(), **own)))
    for n in names:
        assert torch.equal(got[n], want[n])
        if n in own:
            assert got[n] is own[n]
    with pytest.raises(ValueError, match="positions"):
        ds.dflash_block_tables(*args(), positions=torch.zeros(54, dtype=torch.int32, device=dev))
    assert ds.dflash_device_status(clear=True) == 0


@pytest.mark.gpu
def test_tables_of_nearly_two_to_the_31_pages(dev):
    """Fresh pages up to the end of 31 bits: a table and a free list of 8.6 GB each."""
    R, width = 16384, 131071
    if torch.cuda.mem_get_info(dev)[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB of device memory")
    i32 = dict(dtype=torch.int32, device=dev)
    free = torch.arange(R * width, **i32)
    table = torch.full((R, width), -1, **i32)
    zero, new = torch.zeros(R, **i32), torch.full((R,), width, **i32)
    start, kv, held, _, _, needed = ds.dflash_block_tables(zero, new, zero.clone(), free, table, 1, 0)
    # there is no room for the tokens, which only positions and slots need
    assert ds.dflash_device_status(clear=True) == ds.DEVICE_BAD_LENGTH
    assert int(needed) == R * width and (kv == width).all() and (held == width).all()
    assert torch.equal(start.long(), torch.arange(R + 1, device=dev) * width)
    assert torch.equal(table.view(-1), free)


def test_integers_past_31_bits(monkeypatch):
    """A window wider than any context has no bound; sizes that do not fit the C interface are
    refused. (ctypes would pass the low 32 bits: a window of 2^32 as 0.)"""
    launched = []
    monkeypatch.setattr(ds, "_launch", lambda fn, dev, stream, *a: launched.append(a))
    ds.dflash_paged_attention(**attention_arguments(), window_left=12345, window_right=2 ** 31 - 1)
    at = launched[0].index(12345)
    for wide in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1):
        ds.dflash_paged_attention(**attention_arguments(), window_left=wide, window_right=wide)
        assert launched[-1][at:at + 2] == (-1, -1)
    assert launched[0][at:at + 2] == (12345, 2 ** 31 - 1)
    n = len(launched)
    for name in ("page_size", "T"):
        with pytest.raises(ValueError, match=name):
            ds.dflash_block_tables(**{**table_arguments(), name: 2 ** 32 + 16})
    assert len(launched) == n
