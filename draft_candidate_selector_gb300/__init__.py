"""GB300-native DFlash2 low-rank candidate selector.

This is the Python binding of libdflash_gb300.so, whose C ABI is in include/dflash.h.
The functions here marshal torch CUDA tensors into pointers and sizes and allocate any
outputs the caller did not pass. Every step of the method runs in the library's
sm_103a kernels, on the current CUDA stream of the tensors' device or on the stream passed
as `stream`. What a call allocates belongs to the stream it runs on. To order that stream
behind the work that makes the inputs, and to keep the inputs until it has read them, is the
caller's part.

Method (page "vllm.models.beam.nvidia.dflash2"): for request r and step p,
  1. cand_ids, unary = top-K of logits[r, p]        (compute_candidates)
  2. h[r, p] = W_proj . hidden[r, p]                (DFlash2BeamCandidateSelector.hidden_projection)
  3. E[r,p,q,c] = unary[r,p,c]
                  + <pred_cb[cand[r,p-1,q]] * h[r,p], succ_cb[cand[r,p,c]]>
     with the anchor token as the predecessor at p = 0 (DFlash2BeamCandidateSelector)
"""

from __future__ import annotations

import ctypes

import torch

from . import _native
from ._native import (DEVICE_BAD_ID, DEVICE_BAD_LENGTH, DEVICE_NO_PAGES,  # noqa: F401
                      DEVICE_TIMEOUT, DflashError)

__all__ = [
    "dflash_topk_candidates", "dflash_hidden_projection", "dflash_candidate_edges",
    "dflash_selector", "dflash_selector_forward", "dflash_lmhead_topk", "dflash_selector_lmhead",
    "dflash_best_path", "dflash_block_tables", "dflash_store_kv", "dflash_paged_attention",
    "dflash_paged_attention_workspace_bytes",
    "dflash_topk_workspace_bytes",
    "dflash_selector_workspace_bytes", "dflash_lmhead_topk_workspace_bytes",
    "dflash_selector_lmhead_workspace_bytes",
    "dflash_device_status", "dflash_trace_begin", "dflash_trace_end", "DflashError",
    "library_path", "CandidateSelector",
]


def library_path() -> str:
    _native.load()
    return _native._build.LIBRARY


def _stream(dev: torch.device, stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple | None = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(None if t is None else t.data_ptr())


def dflash_topk_workspace_bytes(R: int, S: int, V: int, K: int) -> int:
    """Workspace bytes dflash_topk_candidates needs on the current device (0 = bad sizes)."""
    return int(_native.load().dflash_topk_workspace_bytes(R, S, V, K))


def dflash_selector_workspace_bytes(R: int, S: int, V: int, K: int) -> int:
    return int(_native.load().dflash_selector_workspace_bytes(R, S, V, K))


def dflash_lmhead_topk_workspace_bytes(R: int, S: int, V: int, K: int) -> int:
    return int(_native.load().dflash_lmhead_topk_workspace_bytes(R, S, V, K))


def dflash_selector_lmhead_workspace_bytes(R: int, S: int, V: int, K: int) -> int:
    return int(_native.load().dflash_selector_lmhead_workspace_bytes(R, S, V, K))


def _empty(shape: tuple, dtype: torch.dtype, dev: torch.device, stream,
           handed_out: bool = True) -> torch.Tensor:
    """An output (or, not handed_out, a workspace) of a call on `stream`, None being the current one.

    It comes from the memory of that stream: the allocator takes it back when its last reference
    goes, and must not give it to work that runs beside the call's kernels, nor take it from work
    that still runs on the current stream. What is handed out is kept from that stream, too, until
    the work that the current stream has been given by then is done.
    """
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev.index):
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
    here = torch.cuda.current_stream(dev)
    if dev.index == torch.cuda.current_device():
        torch.cuda.set_stream(stream)          # half of what the context manager costs
        try:
            t = torch.empty(shape, dtype=dtype, device=dev)
        finally:
            torch.cuda.set_stream(here)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=dev)
    if handed_out:
        t.record_stream(here)
    return t


def _workspace(nbytes: int, dev: torch.device, workspace: torch.Tensor | None,
               stream) -> torch.Tensor:
    if nbytes <= 0:
        _native.check(_native.DFLASH_INVALID_ARGUMENT)
    if workspace is None:
        return _empty((nbytes,), torch.uint8, dev, stream, handed_out=False)
    return _check_workspace(workspace, dev)


def _check_workspace(workspace: torch.Tensor, dev: torch.device) -> torch.Tensor:
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != dev:
        raise ValueError(f"workspace must be a CUDA tensor on {dev}, not {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def dflash_topk_candidates(logits: torch.Tensor, K: int, cand_ids: torch.Tensor | None = None,
                           unary: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None,
                           softcap: float = 0.0, scale: float = 1.0):
    """Top-K candidate ids (int32) and their logits (fp32) of logits [R, S, V] fp32.

    softcap and scale are the logits processor's options: the reported values are
    scale * softcap * tanh(x / softcap) (no cap when softcap is 0).
    """
    lib = _native.load()
    if logits.dim() != 3:
        raise ValueError("logits must be [R, S, V]")
    _need(logits, "logits", torch.float32)
    R, S, V = logits.shape
    dev = logits.device
    with torch.cuda.device(dev):
        if cand_ids is None:
            cand_ids = _empty((R, S, K), torch.int32, dev, stream)
        if unary is None:
            unary = _empty((R, S, K), torch.float32, dev, stream)
        _need(cand_ids, "cand_ids", torch.int32, (R, S, K))
        _need(unary, "unary", torch.float32, (R, S, K))
        ws = _workspace(lib.dflash_topk_workspace_bytes(R, S, V, K), dev, workspace, stream)
        _native.check(lib.dflash_topk_candidates(
            _ptr(logits), R, S, V, K, float(softcap), float(scale), _ptr(cand_ids), _ptr(unary),
            _ptr(ws), ws.nbytes, _stream(dev, stream)))
    return cand_ids, unary


def dflash_lmhead_topk(hidden: torch.Tensor, lm_head: torch.Tensor, K: int,
                       cand_ids: torch.Tensor | None = None, unary: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None,
                       softcap: float = 0.0, scale: float = 1.0):
    """Top-K candidates of hidden [R, S, H] . lm_head [V, H]^T without materialised logits."""
    lib = _native.load()
    if hidden.dim() != 3 or lm_head.dim() != 2:
        raise ValueError("hidden must be [R, S, H] and lm_head [V, H]")
    R, S, H = hidden.shape
    V = lm_head.shape[0]
    _need(hidden, "hidden", torch.bfloat16)
    _need(lm_head, "lm_head", torch.bfloat16, (V, H))
    dev = hidden.device
    with torch.cuda.device(dev):
        if cand_ids is None:
            cand_ids = _empty((R, S, K), torch.int32, dev, stream)
        if unary is None:
            unary = _empty((R, S, K), torch.float32, dev, stream)
        _need(cand_ids, "cand_ids", torch.int32, (R, S, K))
        _need(unary, "unary", torch.float32, (R, S, K))
        ws = _workspace(lib.dflash_lmhead_topk_workspace_bytes(R, S, V, K), dev, workspace, stream)
        _native.check(lib.dflash_lmhead_topk(
            _ptr(hidden), _ptr(lm_head), R, S, H, V, K, float(softcap), float(scale),
            _ptr(cand_ids), _ptr(unary), _ptr(ws), ws.nbytes, _stream(dev, stream)))
    return cand_ids, unary


def dflash_hidden_projection(hidden: torch.Tensor, w_proj: torch.Tensor,
                             h_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [R, S, rank] bf16 = hidden [R, S, H] bf16 . w_proj [rank, H]^T (fp32 accumulate)."""
    lib = _native.load()
    if hidden.dim() != 3 or w_proj.dim() != 2:
        raise ValueError("hidden must be [R, S, H] and w_proj [rank, H]")
    R, S, H = hidden.shape
    rank = w_proj.shape[0]
    _need(hidden, "hidden", torch.bfloat16)
    _need(w_proj, "w_proj", torch.bfloat16, (rank, H))
    dev = hidden.device
    with torch.cuda.device(dev):
        if h_out is None:
            h_out = _empty((R, S, rank), torch.bfloat16, dev, stream)
        _need(h_out, "h_out", torch.bfloat16, (R, S, rank))
        _native.check(lib.dflash_hidden_projection(
            _ptr(hidden), _ptr(w_proj), R, S, H, rank, _ptr(h_out), _stream(dev, stream)))
    return h_out


def dflash_candidate_edges(pred_cb: torch.Tensor, succ_cb: torch.Tensor,
                           cand_ids: torch.Tensor, unary: torch.Tensor, h: torch.Tensor,
                           anchors: torch.Tensor, edges: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """Edge scores E [R, S, K, K] fp32 (q = predecessor index, c = candidate index)."""
    lib = _native.load()
    if cand_ids.dim() != 3:
        raise ValueError("cand_ids must be [R, S, K]")
    R, S, K = cand_ids.shape
    V, rank = pred_cb.shape
    _need(pred_cb, "pred_cb", torch.bfloat16, (V, rank))
    _need(succ_cb, "succ_cb", torch.bfloat16, (V, rank))
    _need(cand_ids, "cand_ids", torch.int32)
    _need(unary, "unary", torch.float32, (R, S, K))
    _need(h, "h", torch.bfloat16, (R, S, rank))
    _need(anchors, "anchors", torch.int32, (R,))
    dev = cand_ids.device
    with torch.cuda.device(dev):
        if edges is None:
            edges = _empty((R, S, K, K), torch.float32, dev, stream)
        _need(edges, "edges", torch.float32, (R, S, K, K))
        _native.check(lib.dflash_candidate_edges(
            _ptr(pred_cb), _ptr(succ_cb), _ptr(cand_ids), _ptr(unary), _ptr(h), _ptr(anchors),
            R, S, K, V, rank, _ptr(edges), _stream(dev, stream)))
    return edges


def dflash_selector(logits: torch.Tensor, hidden: torch.Tensor, w_proj: torch.Tensor,
                    pred_cb: torch.Tensor, succ_cb: torch.Tensor, anchors: torch.Tensor,
                    K: int, cand_ids: torch.Tensor | None = None,
                    unary: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                    edges: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None, softcap: float = 0.0, scale: float = 1.0):
    """The whole selector in one library call: returns (cand_ids, unary, h, edges).

    softcap and scale are the logits processor's options (see dflash_topk_candidates).
    """
    lib = _native.load()
    if logits.dim() != 3 or hidden.dim() != 3:
        raise ValueError("logits must be [R, S, V] and hidden [R, S, H]")
    R, S, V = logits.shape
    H = hidden.shape[2]
    rank = w_proj.shape[0]
    _need(logits, "logits", torch.float32)
    _need(hidden, "hidden", torch.bfloat16, (R, S, H))
    _need(w_proj, "w_proj", torch.bfloat16, (rank, H))
    _need(pred_cb, "pred_cb", torch.bfloat16, (V, rank))
    _need(succ_cb, "succ_cb", torch.bfloat16, (V, rank))
    _need(anchors, "anchors", torch.int32, (R,))
    dev = logits.device
    with torch.cuda.device(dev):
        if cand_ids is None:
            cand_ids = _empty((R, S, K), torch.int32, dev, stream)
        if unary is None:
            unary = _empty((R, S, K), torch.float32, dev, stream)
        if h_out is None:
            h_out = _empty((R, S, rank), torch.bfloat16, dev, stream)
        if edges is None:
            edges = _empty((R, S, K, K), torch.float32, dev, stream)
        _need(cand_ids, "cand_ids", torch.int32, (R, S, K))
        _need(unary, "unary", torch.float32, (R, S, K))
        _need(h_out, "h_out", torch.bfloat16, (R, S, rank))
        _need(edges, "edges", torch.float32, (R, S, K, K))
        ws = _workspace(lib.dflash_selector_workspace_bytes(R, S, V, K), dev, workspace, stream)
        _native.check(lib.dflash_selector(
            _ptr(logits), _ptr(hidden), _ptr(w_proj), _ptr(pred_cb), _ptr(succ_cb),
            _ptr(anchors), R, S, K, V, H, rank, float(softcap), float(scale), _ptr(cand_ids),
            _ptr(unary), _ptr(h_out), _ptr(edges), _ptr(ws), ws.nbytes, _stream(dev, stream)))
    return cand_ids, unary, h_out, edges


def dflash_selector_forward(cand_ids: torch.Tensor, unary: torch.Tensor, hidden: torch.Tensor,
                            anchors: torch.Tensor, w_proj: torch.Tensor, pred_cb: torch.Tensor,
                            succ_cb: torch.Tensor, h_out: torch.Tensor | None = None,
                            edges: torch.Tensor | None = None, stream=None):
    """The selector's forward pass on given candidates: returns (h, edges).

    cand_ids int32 [R, S, K] and unary fp32 [R, S, K] are the candidates and their logits;
    h = hidden . w_proj^T is computed first, then the edge scores [R, S, K, K].
    """
    lib = _native.load()
    if cand_ids.dim() != 3 or hidden.dim() != 3:
        raise ValueError("cand_ids must be [R, S, K] and hidden [R, S, H]")
    R, S, K = cand_ids.shape
    H = hidden.shape[2]
    rank = w_proj.shape[0]
    V = pred_cb.shape[0]
    _need(cand_ids, "cand_ids", torch.int32)
    _need(unary, "unary", torch.float32, (R, S, K))
    _need(hidden, "hidden", torch.bfloat16, (R, S, H))
    _need(anchors, "anchors", torch.int32, (R,))
    _need(w_proj, "w_proj", torch.bfloat16, (rank, H))
    _need(pred_cb, "pred_cb", torch.bfloat16, (V, rank))
    _need(succ_cb, "succ_cb", torch.bfloat16, (V, rank))
    dev = hidden.device
    with torch.cuda.device(dev):
        if h_out is None:
            h_out = _empty((R, S, rank), torch.bfloat16, dev, stream)
        if edges is None:
            edges = _empty((R, S, K, K), torch.float32, dev, stream)
        _need(h_out, "h_out", torch.bfloat16, (R, S, rank))
        _need(edges, "edges", torch.float32, (R, S, K, K))
        _native.check(lib.dflash_selector_forward(
            _ptr(cand_ids), _ptr(unary), _ptr(hidden), _ptr(anchors), _ptr(w_proj), _ptr(pred_cb),
            _ptr(succ_cb), R, S, K, V, H, rank, _ptr(h_out), _ptr(edges), _stream(dev, stream)))
    return h_out, edges


def dflash_selector_lmhead(hidden: torch.Tensor, lm_head: torch.Tensor, w_proj: torch.Tensor,
                           pred_cb: torch.Tensor, succ_cb: torch.Tensor, anchors: torch.Tensor,
                           K: int, cand_ids: torch.Tensor | None = None,
                           unary: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                           edges: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None,
                           softcap: float = 0.0, scale: float = 1.0):
    """The draft step from the LM head in one library call: returns (cand_ids, unary, h, edges).

    The candidates come straight from hidden [R, S, H] . lm_head [V, H]^T, as in
    dflash_lmhead_topk; no logits are written.
    """
    lib = _native.load()
    if hidden.dim() != 3 or lm_head.dim() != 2:
        raise ValueError("hidden must be [R, S, H] and lm_head [V, H]")
    R, S, H = hidden.shape
    V = lm_head.shape[0]
    rank = w_proj.shape[0]
    _need(hidden, "hidden", torch.bfloat16)
    _need(lm_head, "lm_head", torch.bfloat16, (V, H))
    _need(w_proj, "w_proj", torch.bfloat16, (rank, H))
    _need(pred_cb, "pred_cb", torch.bfloat16, (V, rank))
    _need(succ_cb, "succ_cb", torch.bfloat16, (V, rank))
    _need(anchors, "anchors", torch.int32, (R,))
    dev = hidden.device
    with torch.cuda.device(dev):
        if cand_ids is None:
            cand_ids = _empty((R, S, K), torch.int32, dev, stream)
        if unary is None:
            unary = _empty((R, S, K), torch.float32, dev, stream)
        if h_out is None:
            h_out = _empty((R, S, rank), torch.bfloat16, dev, stream)
        if edges is None:
            edges = _empty((R, S, K, K), torch.float32, dev, stream)
        _need(cand_ids, "cand_ids", torch.int32, (R, S, K))
        _need(unary, "unary", torch.float32, (R, S, K))
        _need(h_out, "h_out", torch.bfloat16, (R, S, rank))
        _need(edges, "edges", torch.float32, (R, S, K, K))
        ws = _workspace(lib.dflash_selector_lmhead_workspace_bytes(R, S, V, K), dev, workspace, stream)
        _native.check(lib.dflash_selector_lmhead(
            _ptr(hidden), _ptr(lm_head), _ptr(w_proj), _ptr(pred_cb), _ptr(succ_cb),
            _ptr(anchors), R, S, K, V, H, rank, float(softcap), float(scale), _ptr(cand_ids),
            _ptr(unary), _ptr(h_out), _ptr(edges), _ptr(ws), ws.nbytes, _stream(dev, stream)))
    return cand_ids, unary, h_out, edges


def dflash_best_path(edges: torch.Tensor, cand_ids: torch.Tensor, path: torch.Tensor | None = None,
                     tokens: torch.Tensor | None = None, score: torch.Tensor | None = None,
                     stream=None):
    """Max-sum path through edge scores [R, S, K, K]: returns (path int32 [R, S],
    tokens int32 [R, S], score fp32 [R])."""
    lib = _native.load()
    if edges.dim() != 4 or edges.shape[2] != edges.shape[3]:
        raise ValueError("edges must be [R, S, K, K]")
    R, S, K, _ = edges.shape
    _need(edges, "edges", torch.float32)
    _need(cand_ids, "cand_ids", torch.int32, (R, S, K))
    dev = edges.device
    with torch.cuda.device(dev):
        if path is None:
            path = _empty((R, S), torch.int32, dev, stream)
        if tokens is None:
            tokens = _empty((R, S), torch.int32, dev, stream)
        if score is None:
            score = _empty((R,), torch.float32, dev, stream)
        _need(path, "path", torch.int32, (R, S))
        _need(tokens, "tokens", torch.int32, (R, S))
        _need(score, "score", torch.float32, (R,))
        _native.check(lib.dflash_best_path(_ptr(edges), _ptr(cand_ids), R, S, K, _ptr(path),
                                           _ptr(tokens), _ptr(score), _stream(dev, stream)))
    return path, tokens, score


# The calls below are made once per layer or per step of a serving loop, where the host's time
# counts: one comparison decides whether an argument is right, and only a wrong one is looked into
# by _need; addresses go to the library as integers; outputs the caller did not pass are not
# checked, and those of one type share an allocation.

def _checked(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, index: int) -> int:
    """The address of a contiguous tensor of this type and shape on CUDA device `index`."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.shape == shape
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, shape)
    raise _elsewhere(t, name, index)


_INT_MAX = 2 ** 31 - 1      # ctypes passes the low 32 bits of a larger number, without an error


def _elsewhere(t: torch.Tensor, name: str, index: int) -> ValueError:
    return ValueError(f"{name} is on {t.device}, the call's first tensor on cuda:{index}")


def _launch(fn, dev: torch.device, stream, *args) -> None:
    """fn(*args, stream) with dev current."""
    index, current = dev.index, torch.cuda.current_device()
    if index is None:
        index = current
    st = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == current:
        status = fn(*args, st)
    else:
        with torch.cuda.device(index):
            status = fn(*args, st)
    if status:
        _native.check(status)


def dflash_block_tables(context_lens: torch.Tensor, new_lens: torch.Tensor,
                        held_pages: torch.Tensor, free_pages: torch.Tensor,
                        block_table: torch.Tensor, page_size: int, T: int,
                        query_start: torch.Tensor | None = None,
                        kv_lens: torch.Tensor | None = None,
                        held_out: torch.Tensor | None = None,
                        positions: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                        pages_needed: torch.Tensor | None = None, stream=None):
    """One step's block tables and slots: returns (query_start [R + 1], kv_lens [R], held_out [R],
    positions [T], slots [T] int64, pages_needed [1]), all int32 but the slots.

    block_table int32 [R, max_pages] gets each request's new pages, taken in order from
    free_pages; T is the room for new tokens (their number, or more for a padded batch).
    """
    lib = _native._lib or _native.load()
    i32 = torch.int32
    if context_lens.dim() != 1 or free_pages.dim() != 1 or block_table.dim() != 2:
        raise ValueError("context_lens must be [R], free_pages [n], block_table [R, max_pages]")
    (R,), max_pages, n_free = context_lens.shape, block_table.shape[1], free_pages.shape[0]
    if page_size > _INT_MAX or T > _INT_MAX or n_free > _INT_MAX or max_pages > _INT_MAX:
        raise ValueError("page_size, T, max_pages and the number of free pages must be below 2^31")
    dev = context_lens.device
    index = context_lens.get_device()
    if index < 0:
        _need(context_lens, "context_lens", i32)                 # raises
    ctx = _checked(context_lens, "context_lens", i32, (R,), index)
    new = _checked(new_lens, "new_lens", i32, (R,), index)
    held = _checked(held_pages, "held_pages", i32, (R,), index)
    free = _checked(free_pages, "free_pages", i32, (n_free,), index)
    table = _checked(block_table, "block_table", i32, (R, max_pages), index)
    sizes = (R + 1, R, R, T, 1)
    given = (query_start, kv_lens, held_out, positions, pages_needed)
    names = ("query_start", "kv_lens", "held_out", "positions", "pages_needed")
    if given == (None, None, None, None, None):
        room = _empty((3 * R + T + 2,), i32, dev, stream)
        out = room.split_with_sizes(sizes)
        at = room.data_ptr()
        ptrs = (at, at + 4 * (R + 1), at + 4 * (2 * R + 1), at + 4 * (3 * R + 1),
                at + 4 * (3 * R + 1 + T))
    else:
        out = tuple(_empty((n,), i32, dev, stream) if t is None else t
                    for t, n in zip(given, sizes))
        ptrs = tuple(_checked(t, name, i32, (n,), index)
                     for t, name, n in zip(out, names, sizes))
    if slots is None:
        slots = _empty((T,), torch.int64, dev, stream)
        slots_at = slots.data_ptr()
    else:
        slots_at = _checked(slots, "slots", torch.int64, (T,), index)
    _launch(lib.dflash_block_tables, dev, stream, ctx, new, held, free, R, n_free, page_size,
            max_pages, T, table, ptrs[0], ptrs[1], ptrs[2], ptrs[3], slots_at, ptrs[4])
    return out[0], out[1], out[2], out[3], slots, out[4]


_DTYPES = {torch.bfloat16: _native.BF16, torch.float16: _native.FP16,
           torch.float8_e4m3fn: _native.E4M3}


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype | None = None):
    """The type code and strides of a [rows, heads, head_dim] tensor that may be strided in all
    but the last."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] != 1):
        raise ValueError(f"{name} must be [T, heads, head_dim], head_dim contiguous")
    code = _DTYPES.get(t.dtype, _native.E4M3)
    if code == _native.E4M3 or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be bf16 or fp16 (and of one type), got {t.dtype}")
    return code, t.stride()


def _kv_cache(key_cache: torch.Tensor, value_cache: torch.Tensor, k_scale: float,
              v_scale: float, index: int) -> _native.KvCache:
    for t, name in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.get_device() != index:
            raise _elsewhere(t, name, index)
    shape, strides, dtype = key_cache.shape, key_cache.stride(), key_cache.dtype
    if len(shape) != 4 or (strides[3] != 1 and shape[3] != 1):
        raise ValueError("key_cache must be [pages, page_size, kv_heads, head_dim], "
                         "head_dim contiguous")
    if dtype not in _DTYPES:
        raise ValueError(f"key_cache must be bf16, fp16 or float8_e4m3fn, got {dtype}")
    # A dimension of one element may have any stride.
    if (value_cache.shape != shape or value_cache.dtype != dtype
            or (value_cache.stride() != strides
                and any(n != 1 and x != y
                        for n, x, y in zip(shape, strides, value_cache.stride())))):
        raise ValueError("key_cache and value_cache must have one shape, type and strides")
    return _native.KvCache(key_cache.data_ptr(), value_cache.data_ptr(), strides[0], strides[1],
                           strides[2], shape[0], shape[1], shape[2], shape[3], _DTYPES[dtype],
                           k_scale, v_scale)


def dflash_store_kv(key: torch.Tensor, value: torch.Tensor, slots: torch.Tensor,
                    key_cache: torch.Tensor, value_cache: torch.Tensor, k_scale: float = 1.0,
                    v_scale: float = 1.0, stream=None):
    """Store key and value [T, kv_heads, head_dim] (bf16 or fp16, strided views allowed) at slots
    int64 [T] of the caches [pages, page_size, kv_heads, head_dim]: returns (key_cache,
    value_cache). A float8_e4m3fn cache holds x / scale; a negative slot stores nothing.
    """
    lib = _native._lib or _native.load()
    code, ks = _rows(key, "key")
    _, vs = _rows(value, "value", key.dtype)
    index = key.get_device()
    if value.get_device() != index:
        raise _elsewhere(value, "value", index)
    cache = _kv_cache(key_cache, value_cache, k_scale, v_scale, index)
    shape = key.shape
    T = shape[0]
    if shape != (T, cache.kv_heads, cache.head_dim) or value.shape != shape:
        raise ValueError(f"key and value must be [T, {cache.kv_heads}, {cache.head_dim}], got "
                         f"{tuple(key.shape)} and {tuple(value.shape)}")
    at = _checked(slots, "slots", torch.int64, (T,), index)
    _launch(lib.dflash_store_kv, key.device, stream, key.data_ptr(), value.data_ptr(), code, at, T,
            ks[0], ks[1], vs[0], vs[1], cache)
    return key_cache, value_cache


def dflash_paged_attention_workspace_bytes(R: int, T: int, q_heads: int, kv_heads: int,
                                           head_dim: int) -> int:
    return int(_native.load().dflash_paged_attention_workspace_bytes(R, T, q_heads, kv_heads,
                                                                     head_dim))


_workspace_sizes: dict = {}


def _attention_workspace(dev: torch.device, head_dim: int) -> int:
    """The workspace bytes of any call with this head_dim on a device: they depend on nothing else."""
    nbytes = _workspace_sizes.get((dev, head_dim), 0)
    if nbytes == 0:
        with torch.cuda.device(dev):
            nbytes = dflash_paged_attention_workspace_bytes(1, 1, 1, 1, head_dim)
        if nbytes == 0:
            _native.check(_native.DFLASH_INVALID_ARGUMENT)
        _workspace_sizes[(dev, head_dim)] = nbytes
    return nbytes


def dflash_paged_attention(query: torch.Tensor, key_cache: torch.Tensor,
                           value_cache: torch.Tensor, block_table: torch.Tensor,
                           query_start: torch.Tensor, kv_lens: torch.Tensor,
                           scale: float | None = None, window_left: int = -1,
                           window_right: int = 0, softcap: float = 0.0, k_scale: float = 1.0,
                           v_scale: float = 1.0, out: torch.Tensor | None = None,
                           lse: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None):
    """Attention of new tokens over the paged cache, which holds their own keys and values too:
    returns (out [T, q_heads, head_dim], lse fp32 [T, q_heads]).

    query [T, q_heads, head_dim] bf16 or fp16 (strided views allowed); the caches [pages,
    page_size, kv_heads, head_dim] of its type or float8_e4m3fn, in any order of page rows and
    heads; block_table int32 [R, max_pages], query_start int32 [R + 1] and kv_lens int32 [R] as
    dflash_block_tables gives them. A token at position p sees keys p - window_left to
    p + window_right (-1: no bound; window_right 0 is causal). scale defaults to
    1 / sqrt(head_dim).
    """
    lib = _native._lib or _native.load()
    code, qs = _rows(query, "query")
    index = query.get_device()
    cache = _kv_cache(key_cache, value_cache, k_scale, v_scale, index)
    T, Hq, D = query.shape
    if D != cache.head_dim:
        raise ValueError(f"query has head_dim {D}, the cache {cache.head_dim}")
    if block_table.dim() != 2 or kv_lens.dim() != 1:
        raise ValueError("block_table must be [R, max_pages] and kv_lens [R]")
    R, max_pages = block_table.shape
    if window_left > _INT_MAX:                                   # sees all there is
        window_left = -1
    if window_right > _INT_MAX:
        window_right = -1
    table = _checked(block_table, "block_table", torch.int32, (R, max_pages), index)
    start = _checked(query_start, "query_start", torch.int32, (R + 1,), index)
    kv = _checked(kv_lens, "kv_lens", torch.int32, (R,), index)
    dev = query.device
    if out is None:
        out = _empty((T, Hq, D), query.dtype, dev, stream)
        out_at = out.data_ptr()
    else:
        out_at = _checked(out, "out", query.dtype, (T, Hq, D), index)
    if lse is None:
        lse = _empty((T, Hq), torch.float32, dev, stream)
        lse_at = lse.data_ptr()
    else:
        lse_at = _checked(lse, "lse", torch.float32, (T, Hq), index)
    if workspace is None:
        workspace = _empty((_attention_workspace(dev, D),), torch.uint8, dev, stream,
                           handed_out=False)
    else:
        _check_workspace(workspace, dev)
    _launch(lib.dflash_paged_attention, dev, stream, query.data_ptr(), code, T, Hq, qs[0], qs[1],
            cache, table, R, max_pages, start, kv, D ** -0.5 if scale is None else scale,
            window_left, window_right, softcap, out_at, lse_at, workspace.data_ptr(),
            workspace.nbytes)
    return out, lse


def dflash_device_status(clear: bool = True) -> int:
    """DEVICE_* bits set by kernels on the current device since the last clear."""
    flags = ctypes.c_uint32(0)
    _native.check(_native.load().dflash_device_status(ctypes.byref(flags), int(clear)))
    return int(flags.value)


def dflash_trace_begin(n_calls: int) -> None:
    """Record stage timing events for the next n_calls dflash_selector(_lmhead) calls."""
    _native.check(_native.load().dflash_trace_begin(int(n_calls)))


def dflash_trace_end(max_calls: int) -> list[tuple[float, float, float]]:
    """Per traced call: (projection ms, top-k ms, edges ms). Ends the trace."""
    buf = (ctypes.c_float * (3 * max(1, max_calls)))()
    n = ctypes.c_int(0)
    _native.check(_native.load().dflash_trace_end(buf, int(max_calls), ctypes.byref(n)))
    return [(buf[3 * i], buf[3 * i + 1], buf[3 * i + 2]) for i in range(n.value)]


from .selector import CandidateSelector  # noqa: E402  (uses the functions above)
