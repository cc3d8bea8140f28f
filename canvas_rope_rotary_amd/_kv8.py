"""ctypes binding of the 8-bit paged K/V cache: append, attention, pages (see include/mrope.h)."""
from __future__ import annotations

from array import array

import torch

from . import _lib
from ._lib import ROT_DIM, _DTYPES, _invoke, _on_device, load

PAGES_NOT_ENOUGH = 1
PAGES_BAD_ROW = 2
_F8 = torch.float8_e4m3fn
_stream_of = torch._C._cuda_getCurrentRawStream

# The checks below read each property of a tensor once and pass plain integers on: for a decode step of
# few sequences the host's part of a call is most of its time.


def _same_device(first, *others) -> torch.device:
    index = first.get_device()
    if index < 0:
        raise ValueError("all tensors must be on a CUDA (HIP) device")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on the same CUDA (HIP) device")
    return first.device


def _i32(t, name: str, n: int | None = None) -> int:
    """Address of a contiguous int32 vector (of n entries)."""
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor" + ("" if n is None else f" of {n} entries"))
    return t.data_ptr()


def _heads(t, name: str, dtype=None, tokens=None, dim=None):
    """(address, token stride, head stride, heads, tokens, head_dim) of [tokens, heads, head_dim]."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    n, h, d = shape
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must have q's dtype")
    if (tokens is not None and n != tokens) or (dim is not None and d != dim):
        raise ValueError(f"{name} must have q's tokens and head_dim")
    if n * h * d == 0:  # no elements: strides are free
        return t.data_ptr(), h * d, d, h, n, d
    if stride[2] != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    return t.data_ptr(), stride[0], stride[1], h, n, d


def _code(t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return code


def _scratch(nbytes: int, device, workspace=None):
    """(address, bytes, tensor to keep) of a call's workspace: the caller's, else memory of this call from
    torch's allocator.  Calls of their own streams and captured graphs so never share one (memory
    allocated under capture belongs to the graph), and a prepared call keeps its own."""
    if nbytes == 0:
        return None, 0, None
    if workspace is not None:
        if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous() or workspace.device != device:
            raise ValueError("workspace must be a contiguous 1-D uint8 tensor on the call's device")
        return workspace.data_ptr(), workspace.numel(), workspace
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if _lib._recording is not None:
        _lib._held.append(t)
    return t.data_ptr(), nbytes, t


def _tables(t, n: int | None = None):
    """(address, row stride, width, rows) of the block tables."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 2 or (n is not None and shape[0] != n) or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("block_tables must be an int32 [n, width] tensor with unit column stride" + ("" if n is None else f" and n = {n}"))
    return t.data_ptr(), max(t.stride(0), shape[1]) if shape[0] < 2 else t.stride(0), shape[1]


def _kv8(k_cache, v_cache, k_scale, v_scale, nk: int | None, D: int):
    """Check an 8-bit cache pair with its scales; returns the C arguments."""
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[3] != D or (nk is not None and shape[2] != nk) or stride[3] != 1:
        raise ValueError("k_cache must be [num_blocks, block_size, n_kv_heads, head_dim] with q's head_dim")
    for c, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if c.dtype is not _F8 and c.dtype is not torch.uint8:
            raise ValueError(f"{name} must be float8_e4m3fn (or its codes in uint8)")
    if v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError("v_cache must have k_cache's shape and strides")
    blocks, bs, nk, _ = shape
    for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if s.dtype is not torch.float32 or s.shape != (blocks, nk) or not s.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 [num_blocks, n_kv_heads] tensor")
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), bs, blocks, stride[0], stride[1],
            stride[2])


def apply_kv8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, planes_: torch.Tensor, cu_seqlens: torch.Tensor,
              block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
              v_scale: torch.Tensor, theta: float = 1e7, *, pos_offset: torch.Tensor | None = None,
              rot_dim: int = ROT_DIM):
    """apply_kv for a cache held in 8 bits: q [T, Hq, D] rotated in place; k [T, Hk, D] rotated and v
    copied into k_cache / v_cache [num_blocks, block_size, Hk, D] (float8_e4m3fn) with one power-of-two
    scale for each page and head in k_scale / v_scale [num_blocks, Hk].  Token i of sequence s
    (cu_seqlens) goes to position pos_offset[s] + i (None: 0), in the page that block_tables
    [n, width] names for it; a page outside the pool is skipped.  Returns (q, k_cache, v_cache)."""
    dev = _same_device(q, k, v, planes_, cu_seqlens, block_tables, k_cache, v_cache, k_scale, v_scale, pos_offset)
    dt = _code(q)
    qp, qt, qh, nq, T, D = _heads(q, "q")
    kp, kt, kh, nk, _, _ = _heads(k, "k", q.dtype, T, D)
    vp, vt, vh, nv, _, _ = _heads(v, "v", q.dtype, T, D)
    if nv != nk:
        raise ValueError("v must have k's heads")
    if planes_.dtype is not torch.int32 or planes_.dim() != 2 or planes_.shape[0] != 3 or planes_.shape[1] < T \
            or planes_.stride(1) != 1:
        raise ValueError("planes must be an int32 [3, >= tokens] tensor with unit column stride")
    cu = _i32(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    off = None if pos_offset is None else _i32(pos_offset, "pos_offset", n)
    cache = _kv8(k_cache, v_cache, k_scale, v_scale, nk, D)
    with _on_device(dev):
        _invoke(load().mrope_apply_kv8, qp, qt, qh, nq, kp, kt, kh, nk, vp, vt, vh, T, D, rot_dim, dt, planes_.data_ptr(),
                planes_.stride(0), float(theta), cu, n, off, *_tables(block_tables, n), *cache, _stream_of(dev.index))
    return q, k_cache, v_cache


def decode_kv8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, amount: torch.Tensor,
               block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, theta: float = 1e7, *, rot_dim: int = ROT_DIM):
    """decode for a cache held in 8 bits: one new token a sequence, rotated at plane pos - amount and
    written at position pos of its sequence (see apply_kv8).  Returns (q, k_cache, v_cache)."""
    dev = _same_device(q, k, v, pos, amount, block_tables, k_cache, v_cache, k_scale, v_scale)
    dt = _code(q)
    qp, qt, qh, nq, n, D = _heads(q, "q")
    kp, kt, kh, nk, _, _ = _heads(k, "k", q.dtype, n, D)
    vp, vt, vh, nv, _, _ = _heads(v, "v", q.dtype, n, D)
    if nv != nk:
        raise ValueError("v must have k's heads")
    cache = _kv8(k_cache, v_cache, k_scale, v_scale, nk, D)
    with _on_device(dev):
        _invoke(load().mrope_decode_kv8, qp, qt, qh, nq, kp, kt, kh, nk, vp, vt, vh, n, _i32(pos, "pos", n),
                _i32(amount, "amount", n), *_tables(block_tables, n), *cache, D, rot_dim, dt, float(theta),
                _stream_of(dev.index))
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
    dev = _same_device(q, cu_seqlens, context_lens, block_tables, k_cache, v_cache, k_scale, v_scale, out, lse, workspace)
    dt = _code(q)
    qp, qt, qh, nq, T, D = _heads(q, "q")
    cu, n = None, T
    if cu_seqlens is not None:
        cu = _i32(cu_seqlens, "cu_seqlens")
        n = cu_seqlens.numel() - 1
    ctx = _i32(context_lens, "context_lens", n)
    cache = _kv8(k_cache, v_cache, k_scale, v_scale, None, D)
    nk, bs, blocks = k_cache.shape[2], cache[4], cache[5]
    if out is None:
        out = torch.empty((T, nq, D), dtype=q.dtype, device=dev)
    op, ot, oh, no, _, _ = _heads(out, "out", q.dtype, T, D)
    if no != nq:
        raise ValueError("out must have q's shape")
    if lse is None and return_lse:
        lse = torch.empty((T, nq), dtype=torch.float32, device=dev)
    if lse is not None and (lse.shape != (T, nq) or lse.dtype is not torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor")
    tp, ts, tw = _tables(block_tables, n)
    lib = load()
    need = lib.mrope_attend_kv8_workspace_bytes(T, n, nq, nk, D, dt, cu is None, tw if blocks else 0, bs)
    with _on_device(dev):
        ws, ws_bytes, keep = _scratch(need, dev, workspace)
        _invoke(lib.mrope_attend_kv8, qp, qt, qh, nq, T, nk, D, dt, cu, n, ctx, tp, ts, tw, *cache,
                D ** -0.5 if softmax_scale is None else float(softmax_scale), op, ot, oh,
                None if lse is None else lse.data_ptr(), ws, ws_bytes, _stream_of(dev.index))
    return out, lse


def attend_kv8_workspace_bytes(q: torch.Tensor, n_seqs: int, block_tables: torch.Tensor, k_cache: torch.Tensor,
                               one_token: bool) -> int:
    """Bytes of attend_kv8's workspace for these shapes (one_token: cu_seqlens is None)."""
    return int(load().mrope_attend_kv8_workspace_bytes(q.shape[0], int(n_seqs), q.shape[1], k_cache.shape[2], q.shape[2],
                                                       _code(q), int(one_token),
                                                       block_tables.shape[1] if k_cache.shape[0] else 0, k_cache.shape[1]))


# ---------------------------------------------------------------- pages -------------------------
def _state(refcount, block_tables, seq_lens):
    rows = block_tables.shape[0]
    return (_i32(refcount, "refcount"), refcount.numel(), *_tables(block_tables), _i32(seq_lens, "seq_lens", rows), rows)


def _pools(pools, n_pages: int):
    """The pools as an array of mrope_pool (address, bytes of a page, bytes from page to page)."""
    flat = []
    for i, t in enumerate(pools):
        shape = t.shape
        if not shape or shape[0] != n_pages:
            raise ValueError(f"pool {i} must have one entry a page ({n_pages})")
        if n_pages == 0:
            flat += (0, 1, 1)
            continue
        numel, item = t.numel() // n_pages, t.element_size()
        step = numel
        if not t.is_contiguous():
            stride, want = t.stride(), 1
            for k in range(len(shape) - 1, 0, -1):
                if shape[k] > 1 and stride[k] != want:
                    raise ValueError(f"pool {i}: a page must be contiguous")
                want *= shape[k]
            step = stride[0] if n_pages > 1 else numel
        if numel == 0 or step < numel:
            raise ValueError(f"pool {i}: pages are empty or overlap")
        flat += (t.data_ptr(), numel * item, step * item)
    arr = array("q", flat or (0, 0, 0))
    if _lib._recording is not None:
        _lib._held.append(arr)
    return arr, len(pools)


def _pages_ws(refcount, block_tables, dev, workspace):
    return _scratch(load().mrope_pages_workspace_bytes(refcount.numel(), block_tables.shape[0]), dev, workspace)


def _i32_out(t, name, n, dev):
    if t is None:
        return torch.empty(n, dtype=torch.int32, device=dev)
    _i32(t, name, n)
    return t


def pages_grow(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, rows: torch.Tensor,
               new_lens: torch.Tensor, block_size: int, *, status: torch.Tensor | None = None, workspace=None):
    """Give rows[i] of block_tables pages for new_lens[i] positions, lowest free page first, and set its
    length.  refcount [num_blocks], block_tables [n_rows, width] (-1: no page) and seq_lens [n_rows] are
    the state, all int32.  Returns status int32 [n]: 0, PAGES_NOT_ENOUGH or PAGES_BAD_ROW."""
    dev = _same_device(refcount, block_tables, seq_lens, rows, new_lens, status, workspace)
    state = _state(refcount, block_tables, seq_lens)
    rp, n = _i32(rows, "rows"), rows.numel()
    lp = _i32(new_lens, "new_lens", n)
    status = _i32_out(status, "status", n, dev)
    with _on_device(dev):
        ws, ws_bytes, keep = _pages_ws(refcount, block_tables, dev, workspace)
        _invoke(load().mrope_pages_grow, *state, int(block_size), rp, lp, n, status.data_ptr(), ws, ws_bytes, _stream_of(dev.index))
    return status


def pages_free(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, rows: torch.Tensor):
    """Empty the rows: each of their pages loses a reference (0 = free)."""
    dev = _same_device(refcount, block_tables, seq_lens, rows)
    state = _state(refcount, block_tables, seq_lens)
    rp = _i32(rows, "rows")
    with _on_device(dev):
        _invoke(load().mrope_pages_free, *state, rp, rows.numel(), _stream_of(dev.index))


def pages_fork(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor, block_size: int, pools, *, status: torch.Tensor | None = None, workspace=None):
    """Make each empty row dst[i] a copy of row src[i]: full pages are shared, a last page that is not
    full is copied in every tensor of `pools` (one entry a page: caches and scales of any layers).
    Returns status as pages_grow."""
    dev = _same_device(refcount, block_tables, seq_lens, src, dst, status, workspace, *pools)
    state = _state(refcount, block_tables, seq_lens)
    sp, n = _i32(src, "src"), src.numel()
    dp = _i32(dst, "dst", n)
    arr, n_pools = _pools(pools, state[1])
    status = _i32_out(status, "status", n, dev)
    with _on_device(dev):
        ws, ws_bytes, keep = _pages_ws(refcount, block_tables, dev, workspace)
        _invoke(load().mrope_pages_fork, *state, int(block_size), sp, dp, n, status.data_ptr(), arr.buffer_info()[0], n_pools,
                ws, ws_bytes, _stream_of(dev.index))
    return status


def pages_compact(refcount: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, pools, *,
                  moved: torch.Tensor | None = None, workspace=None):
    """Move the live pages to the lowest indexes, in every tensor of `pools` and in the tables.  Returns
    moved int32 [1]: how many pages moved."""
    dev = _same_device(refcount, block_tables, seq_lens, moved, workspace, *pools)
    state = _state(refcount, block_tables, seq_lens)
    arr, n_pools = _pools(pools, state[1])
    moved = _i32_out(moved, "moved", 1, dev)
    with _on_device(dev):
        ws, ws_bytes, keep = _pages_ws(refcount, block_tables, dev, workspace)
        _invoke(load().mrope_pages_compact, *state, moved.data_ptr(), arr.buffer_info()[0], n_pools, ws, ws_bytes,
                _stream_of(dev.index))
    return moved


def pages_copy(src: torch.Tensor, dst: torch.Tensor, pools):
    """Copy page src[i] to page dst[i] in every tensor of `pools`.  A page may be many pairs' source, but
    one pair's destination only and not both."""
    if not pools:
        raise ValueError("pools is empty")
    dev = _same_device(src, dst, *pools)
    sp, n = _i32(src, "src"), src.numel()
    dp = _i32(dst, "dst", n)
    arr, n_pools = _pools(pools, pools[0].shape[0])
    with _on_device(dev):
        _invoke(load().mrope_pages_copy, arr.buffer_info()[0], n_pools, pools[0].shape[0], sp, dp, n, _stream_of(dev.index))
