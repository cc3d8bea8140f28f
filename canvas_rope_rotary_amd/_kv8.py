"""ctypes binding of the 8-bit paged K/V cache: append, attention, pages (see include/mrope.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import ROT_DIM, MropePool, _dtype_code, _heads, _i32_vec, _invoke, _on_device, _ptr, _qk_args, _require_cuda, _stream, load

PAGES_NOT_ENOUGH = 1
PAGES_BAD_ROW = 2


def _scratch(nbytes: int, device, workspace=None):
    """Workspace of one call: the caller's, else memory of this call from torch's allocator.  Calls of
    their own streams and captured graphs so never share one (memory allocated under capture belongs to
    the graph), and a prepared call keeps its own."""
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous() or workspace.device != device:
            raise ValueError("workspace must be a contiguous 1-D uint8 tensor on the call's device")
        return workspace, workspace.numel()
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if _lib._recording is not None:
        _lib._held.append(t)
    return t, nbytes


def _tables(t: torch.Tensor, n: int | None = None):
    if t.dtype != torch.int32 or t.dim() != 2 or (n is not None and t.shape[0] != n) or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("block_tables must be an int32 [n, width] tensor with unit column stride" + ("" if n is None else f" and n = {n}"))
    return _ptr(t), t.stride(0), t.shape[1]


def _kv8(k_cache, v_cache, k_scale, v_scale, nk: int | None, D: int):
    """Check an 8-bit cache pair with its scales; returns (KV heads, the C arguments)."""
    for c, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if c.dim() != 4 or c.shape[3] != D or (nk is not None and c.shape[2] != nk) or c.stride(3) != 1 \
                or c.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError(f"{name} must be [num_blocks, block_size, n_kv_heads, head_dim], float8_e4m3fn (or its codes in uint8)")
    if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("v_cache must have k_cache's shape and strides")
    nk = k_cache.shape[2]
    for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if s.dtype != torch.float32 or s.shape != (k_cache.shape[0], nk) or not s.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 [num_blocks, n_kv_heads] tensor")
    return nk, (_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), k_cache.shape[1], k_cache.shape[0],
                k_cache.stride(0), k_cache.stride(1), k_cache.stride(2))


def _v_args(v, k, what):
    vt, vh, nv, Dv = _heads(v, "v")
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError(f"{what}: v must match k's shape and dtype")
    return _ptr(v), vt, vh


def apply_kv8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, planes_: torch.Tensor, cu_seqlens: torch.Tensor,
              block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
              v_scale: torch.Tensor, theta: float = 1e7, *, pos_offset: torch.Tensor | None = None,
              rot_dim: int = ROT_DIM):
    """apply_kv for a cache held in 8 bits: q [T, Hq, D] rotated in place; k [T, Hk, D] rotated and v
    copied into k_cache / v_cache [num_blocks, block_size, Hk, D] (float8_e4m3fn) with one power-of-two
    scale for each page and head in k_scale / v_scale [num_blocks, Hk].  Token i of sequence s
    (cu_seqlens) goes to position pos_offset[s] + i (None: 0), in the page that block_tables
    [n, width] names for it; a page outside the pool is skipped.  Returns (q, k_cache, v_cache)."""
    dev = _require_cuda(q, k, v, planes_, cu_seqlens, block_tables, k_cache, v_cache, k_scale, v_scale, pos_offset)
    dt, qt, qh, nq, kt, kh, nk, D = _qk_args(q, k, None, None)
    T = q.shape[0]
    if planes_.dtype != torch.int32 or planes_.dim() != 2 or planes_.shape[0] != 3 or planes_.shape[1] < T \
            or planes_.stride(1) != 1:
        raise ValueError("planes must be an int32 [3, >= tokens] tensor with unit column stride")
    _i32_vec(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    if pos_offset is not None:
        _i32_vec(pos_offset, "pos_offset", n)
    vp = _v_args(v, k, "apply_kv8")
    _, cache = _kv8(k_cache, v_cache, k_scale, v_scale, nk, D)
    with _on_device(dev):
        _invoke(load().mrope_apply_kv8, _ptr(q), qt, qh, nq, _ptr(k), kt, kh, nk, *vp, T, D, rot_dim, dt, _ptr(planes_),
                planes_.stride(0), float(theta), _ptr(cu_seqlens), n, _ptr(pos_offset), *_tables(block_tables, n), *cache,
                _stream(dev))
    return q, k_cache, v_cache


def decode_kv8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, amount: torch.Tensor,
               block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, theta: float = 1e7, *, rot_dim: int = ROT_DIM):
    """decode for a cache held in 8 bits: one new token a sequence, rotated at plane pos - amount and
    written at position pos of its sequence (see apply_kv8).  Returns (q, k_cache, v_cache)."""
    dev = _require_cuda(q, k, v, pos, amount, block_tables, k_cache, v_cache, k_scale, v_scale)
    dt, qt, qh, nq, kt, kh, nk, D = _qk_args(q, k, None, None)
    n = q.shape[0]
    _i32_vec(pos, "pos", n)
    _i32_vec(amount, "amount", n)
    vp = _v_args(v, k, "decode_kv8")
    _, cache = _kv8(k_cache, v_cache, k_scale, v_scale, nk, D)
    with _on_device(dev):
        _invoke(load().mrope_decode_kv8, _ptr(q), qt, qh, nq, _ptr(k), kt, kh, nk, *vp, n, _ptr(pos), _ptr(amount),
                *_tables(block_tables, n), *cache, D, rot_dim, dt, float(theta), _stream(dev))
    return q, k_cache, v_cache


def attend_kv8(q: torch.Tensor, cu_seqlens: torch.Tensor | None, context_lens: torch.Tensor, block_tables: torch.Tensor,
               k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, *,
               softmax_scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               return_lse: bool = False, workspace: torch.Tensor | None = None):
    """Causal attention of rotated query tokens q [T, Hq, D] over the 8-bit paged cache.  cu_seqlens
    [n + 1] gives the query tokens of each sequence (None: one each); they are the last of its
    context_lens [n] positions, and token i of len sees the positions up to context - len + i.
    softmax_scale: None = D ** -0.5.  out [T, Hq, D] of q's dtype and lse [T, Hq] float32 (natural
    logarithm) are allocated where they are not given; a row that sees nothing is 0, its lse -inf.
    workspace: uint8 memory for a caller that allocates nothing (attend_kv8_workspace_bytes).
    Returns (out, lse or None)."""
    dev = _require_cuda(q, cu_seqlens, context_lens, block_tables, k_cache, v_cache, k_scale, v_scale, out, lse, workspace)
    dt = _dtype_code(q)
    qt, qh, nq, D = _heads(q, "q")
    T = q.shape[0]
    if cu_seqlens is not None:
        _i32_vec(cu_seqlens, "cu_seqlens")
        n = cu_seqlens.numel() - 1
    else:
        n = T
    _i32_vec(context_lens, "context_lens", n)
    nk, cache = _kv8(k_cache, v_cache, k_scale, v_scale, None, D)
    if out is None:
        out = torch.empty((T, nq, D), dtype=q.dtype, device=dev)
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and dtype")
    ot, oh, _, _ = _heads(out, "out")
    if lse is None and return_lse:
        lse = torch.empty((T, nq), dtype=torch.float32, device=dev)
    if lse is not None and (lse.shape != (T, nq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor")
    tp, ts, tw = _tables(block_tables, n)
    need = int(load().mrope_attend_kv8_workspace_bytes(T, n, nq, nk, D, dt, int(cu_seqlens is None),
                                                       tw if k_cache.shape[0] else 0, k_cache.shape[1]))
    with _on_device(dev):
        ws, ws_bytes = _scratch(need, dev, workspace)
        _invoke(load().mrope_attend_kv8, _ptr(q), qt, qh, nq, T, nk, D, dt, _ptr(cu_seqlens), n, _ptr(context_lens),
                tp, ts, tw, *cache, float(D ** -0.5 if softmax_scale is None else softmax_scale), _ptr(out), ot, oh,
                _ptr(lse), _ptr(ws), ws_bytes, _stream(dev))
    return out, lse


def attend_kv8_workspace_bytes(q: torch.Tensor, n_seqs: int, block_tables: torch.Tensor, k_cache: torch.Tensor,
                               one_token: bool) -> int:
    """Bytes of attend_kv8's workspace for these shapes (one_token: cu_seqlens is None)."""
    return int(load().mrope_attend_kv8_workspace_bytes(q.shape[0], int(n_seqs), q.shape[1], k_cache.shape[2], q.shape[2],
                                                       _dtype_code(q), int(one_token),
                                                       block_tables.shape[1] if k_cache.shape[0] else 0, k_cache.shape[1]))


# ---------------------------------------------------------------- pages -------------------------
def _state(refcount, block_tables, seq_lens):
    _i32_vec(refcount, "refcount")
    tp, ts, tw = _tables(block_tables)
    _i32_vec(seq_lens, "seq_lens", block_tables.shape[0])
    return _ptr(refcount), refcount.numel(), tp, ts, tw, _ptr(seq_lens), block_tables.shape[0]


def _pools(pools, n_pages: int):
    a = (MropePool * max(1, len(pools)))()
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != n_pages:
            raise ValueError(f"pool {i} must have one entry a page ({n_pages})")
        inner = t[0] if n_pages else t
        if not inner.is_contiguous() or (n_pages and inner.numel() == 0):
            raise ValueError(f"pool {i}: a page must be contiguous")
        size = max(1, inner.numel() * t.element_size()) if n_pages else 1
        a[i].ptr = t.data_ptr()
        a[i].page_bytes = size
        a[i].page_stride = max(size, t.stride(0) * t.element_size()) if n_pages > 1 else size
        if n_pages > 1 and t.stride(0) * t.element_size() < size:
            raise ValueError(f"pool {i}: pages overlap")
    return a, len(pools)


def _pages_ws(refcount, block_tables, dev, workspace):
    return _scratch(int(load().mrope_pages_workspace_bytes(refcount.numel(), block_tables.shape[0])), dev, workspace)


def pages_grow(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, rows: torch.Tensor,
               new_lens: torch.Tensor, block_size: int, *, status: torch.Tensor | None = None, workspace=None):
    """Give rows[i] of block_tables pages for new_lens[i] positions, lowest free page first, and set its
    length.  refcount [num_blocks], block_tables [n_rows, width] (-1: no page) and seq_lens [n_rows] are
    the state, all int32.  Returns status int32 [n]: 0, PAGES_NOT_ENOUGH or PAGES_BAD_ROW."""
    dev = _require_cuda(refcount, block_tables, seq_lens, rows, new_lens, status, workspace)
    state = _state(refcount, block_tables, seq_lens)
    n = _i32_vec(rows, "rows").numel()
    _i32_vec(new_lens, "new_lens", n)
    status = torch.empty(n, dtype=torch.int32, device=dev) if status is None else _i32_vec(status, "status", n)
    with _on_device(dev):
        ws, ws_bytes = _pages_ws(refcount, block_tables, dev, workspace)
        _invoke(load().mrope_pages_grow, *state, int(block_size), _ptr(rows), _ptr(new_lens), n, _ptr(status), _ptr(ws),
                ws_bytes, _stream(dev))
    return status


def pages_free(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, rows: torch.Tensor):
    """Empty the rows: each of their pages loses a reference (0 = free)."""
    dev = _require_cuda(refcount, block_tables, seq_lens, rows)
    state = _state(refcount, block_tables, seq_lens)
    n = _i32_vec(rows, "rows").numel()
    with _on_device(dev):
        _invoke(load().mrope_pages_free, *state, _ptr(rows), n, _stream(dev))


def pages_fork(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor, block_size: int, pools, *, status: torch.Tensor | None = None, workspace=None):
    """Make each empty row dst[i] a copy of row src[i]: full pages are shared, a last page that is not
    full is copied in every tensor of `pools` (one entry a page: caches and scales of any layers).
    Returns status as pages_grow."""
    dev = _require_cuda(refcount, block_tables, seq_lens, src, dst, status, workspace, *pools)
    state = _state(refcount, block_tables, seq_lens)
    n = _i32_vec(src, "src").numel()
    _i32_vec(dst, "dst", n)
    arr, n_pools = _pools(pools, refcount.numel())
    status = torch.empty(n, dtype=torch.int32, device=dev) if status is None else _i32_vec(status, "status", n)
    with _on_device(dev):
        ws, ws_bytes = _pages_ws(refcount, block_tables, dev, workspace)
        _invoke(load().mrope_pages_fork, *state, int(block_size), _ptr(src), _ptr(dst), n, _ptr(status), arr, n_pools,
                _ptr(ws), ws_bytes, _stream(dev))
    return status


def pages_compact(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, pools, *,
                  moved: torch.Tensor | None = None, workspace=None):
    """Move the live pages to the lowest indexes, in every tensor of `pools` and in the tables.  Returns
    moved int32 [1]: how many pages moved."""
    dev = _require_cuda(refcount, block_tables, seq_lens, moved, workspace, *pools)
    state = _state(refcount, block_tables, seq_lens)
    arr, n_pools = _pools(pools, refcount.numel())
    moved = torch.empty(1, dtype=torch.int32, device=dev) if moved is None else _i32_vec(moved, "moved", 1)
    with _on_device(dev):
        ws, ws_bytes = _pages_ws(refcount, block_tables, dev, workspace)
        _invoke(load().mrope_pages_compact, *state, _ptr(moved), arr, n_pools, _ptr(ws), ws_bytes, _stream(dev))
    return moved


def pages_copy(src: torch.Tensor, dst: torch.Tensor, pools):
    """Copy page src[i] to page dst[i] in every tensor of `pools`.  A page may be many pairs' source, but
    one pair's destination only and not both."""
    if not pools:
        raise ValueError("pools is empty")
    dev = _require_cuda(src, dst, *pools)
    n = _i32_vec(src, "src").numel()
    _i32_vec(dst, "dst", n)
    arr, n_pools = _pools(pools, pools[0].shape[0])
    with _on_device(dev):
        _invoke(load().mrope_pages_copy, arr, n_pools, pools[0].shape[0], _ptr(src), _ptr(dst), n, _stream(dev))
