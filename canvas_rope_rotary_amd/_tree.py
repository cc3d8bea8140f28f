"""ctypes binding of the calls for trees of drafted tokens: planes and masks, attention, verification, and the
accepted path's cache rows (see include/mrope.h)."""
from __future__ import annotations

from array import array

import torch

from . import _lib
from ._kv8 import _code, _heads, _i32, _i32_out, _kv8, _same_device, _scratch, _stream_of, _tables
from ._lib import _invoke, _on_device, load

TREE_MAX_TOKENS = 1024
MAX_LAYERS = 64


def _mask(t, T: int):
    """(address, words) of a mask [tokens, words]."""
    if t.dtype is not torch.int64 or t.dim() != 2 or t.shape[0] != T or not t.is_contiguous():
        raise ValueError("mask must be a contiguous int64 [tokens, words] tensor")
    return t.data_ptr(), t.shape[1]


def _f32(t, name: str, n: int) -> int:
    if t.dtype is not torch.float32 or t.dim() != 1 or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous 1-D float32 tensor of {n} entries")
    return t.data_ptr()


def _rows(t, name: str, dtype, T: int, vocab: int):
    """(address, row stride) of distributions [tokens, vocab]."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have target_probs' dtype")
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] != vocab or (vocab > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [tokens, vocab] with unit column stride")
    return t.data_ptr(), t.stride(0) if T > 1 else vocab


def planes_tree(parents: torch.Tensor, cu_seqlens: torch.Tensor, pos_offset: torch.Tensor, amount: torch.Tensor | None = None, *,
                mask_words: int = 1, planes: torch.Tensor | None = None, mask: torch.Tensor | None = None):
    """Position planes and masks of trees of drafted tokens.  parents [T] int32: each token's parent as an
    index within its sequence (outside [0, i): none); pos_offset [n] int32: the position of each sequence's
    token 0, amount [n] int32 (None: 0).  Returns (planes int32 [3, T]: pos_offset + depth - amount, mask int64
    [T, mask_words]: bit b of word w is set if token 64 w + b of the sequence is the row's token or an ancestor
    of it), for apply_kv8 and attend_tree_kv8 of every layer."""
    dev = _same_device(parents, cu_seqlens, pos_offset, amount, planes, mask)
    T = parents.numel()
    pp, cu = _i32(parents, "parents"), _i32(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    off = _i32(pos_offset, "pos_offset", n)
    am = None if amount is None else _i32(amount, "amount", n)
    if planes is None:
        planes = torch.empty((3, T), dtype=torch.int32, device=dev)
    elif planes.dtype is not torch.int32 or planes.dim() != 2 or planes.shape[0] != 3 or planes.shape[1] < T or planes.stride(1) != 1:
        raise ValueError("planes must be an int32 [3, >= tokens] tensor with unit column stride")
    if mask is None:
        mask = torch.empty((T, int(mask_words)), dtype=torch.int64, device=dev)
    mp, words = _mask(mask, T)
    with _on_device(dev):
        _invoke(load().mrope_planes_tree, pp, T, cu, n, off, am, planes.data_ptr(), planes.stride(0), mp, words,
                _stream_of(dev.index))
    return planes, mask


def attend_tree_kv8(q: torch.Tensor, cu_seqlens: torch.Tensor, context_lens: torch.Tensor, mask: torch.Tensor,
                    block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, *, softmax_scale: float | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None):
    """attend_kv8 under a mask over the query tokens: token i of a sequence of len sees the positions before
    context - len, and those of the sequence's tokens whose bits are set in its row of mask int64 [T, words]
    (see planes_tree).  Everything else as in attend_kv8.  Returns (out, lse or None)."""
    dev = _same_device(q, cu_seqlens, context_lens, mask, block_tables, k_cache, v_cache, k_scale, v_scale, out, lse, workspace)
    dt = _code(q)
    qp, qt, qh, nq, T, D = _heads(q, "q")
    cu = _i32(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    ctx = _i32(context_lens, "context_lens", n)
    mp, words = _mask(mask, T)
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
    need = lib.mrope_attend_tree_kv8_workspace_bytes(T, n, nq, nk, D, dt, tw if blocks else 0, bs)
    with _on_device(dev):
        ws, ws_bytes, keep = _scratch(need, dev, workspace)
        _invoke(lib.mrope_attend_tree_kv8, qp, qt, qh, nq, T, nk, D, dt, cu, n, ctx, mp, words, tp, ts, tw, *cache,
                D ** -0.5 if softmax_scale is None else float(softmax_scale), op, ot, oh,
                None if lse is None else lse.data_ptr(), ws, ws_bytes, _stream_of(dev.index))
    return out, lse


def attend_tree_kv8_workspace_bytes(q: torch.Tensor, n_seqs: int, block_tables: torch.Tensor, k_cache: torch.Tensor) -> int:
    """Bytes of attend_tree_kv8's workspace for these shapes."""
    return int(load().mrope_attend_tree_kv8_workspace_bytes(q.shape[0], int(n_seqs), q.shape[1], k_cache.shape[2], q.shape[2],
                                                            _code(q), block_tables.shape[1] if k_cache.shape[0] else 0,
                                                            k_cache.shape[1]))


def verify_tree(target_probs: torch.Tensor, ids: torch.Tensor, parents: torch.Tensor | None, cu_seqlens: torch.Tensor,
                u_accept: torch.Tensor, u_next: torch.Tensor, *, draft_probs: torch.Tensor | None = None,
                n_kept: torch.Tensor | None = None, path: torch.Tensor | None = None, next_ids: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None):
    """Which drafted tokens the target accepts, and the token after them.  target_probs [T, vocab]: the
    target's distribution after each token; ids [T] int32 and parents [T] int32 the trees (parents None:
    chains); u_accept [T] and u_next [n] float32 random numbers in [0, 1).  draft_probs [T, vocab]: the
    distributions that each token's children were drawn from (None: they were not drawn).  Returns
    (n_kept [n]: accepted tokens, token 0 included; path [T]: their indices in order, then -1; next_ids [n]),
    all int32: n_kept and path are what keep_kv8 takes."""
    dev = _same_device(target_probs, ids, parents, cu_seqlens, u_accept, u_next, draft_probs, n_kept, path, next_ids, workspace)
    dt = _code(target_probs)
    T, vocab = ids.numel(), target_probs.shape[-1]
    ip = _i32(ids, "ids")
    tp, ts = _rows(target_probs, "target_probs", target_probs.dtype, T, vocab)
    dp, ds = (None, 0) if draft_probs is None else _rows(draft_probs, "draft_probs", target_probs.dtype, T, vocab)
    pp = None if parents is None else _i32(parents, "parents", T)
    cu = _i32(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    ua, un = _f32(u_accept, "u_accept", T), _f32(u_next, "u_next", n)
    n_kept, path = _i32_out(n_kept, "n_kept", n, dev), _i32_out(path, "path", T, dev)
    next_ids = _i32_out(next_ids, "next_ids", n, dev)
    lib = load()
    need = lib.mrope_verify_tree_workspace_bytes(n, vocab, dp is not None, pp is not None)
    with _on_device(dev):
        ws, ws_bytes, keep = _scratch(need, dev, workspace)
        _invoke(lib.mrope_verify_tree, tp, ts, dp, ds, vocab, dt, T, ip, pp, cu, n, ua, un, n_kept.data_ptr(), path.data_ptr(),
                next_ids.data_ptr(), ws, ws_bytes, _stream_of(dev.index))
    return n_kept, path, next_ids


def keep_kv8(n_kept: torch.Tensor, path: torch.Tensor, cu_seqlens: torch.Tensor, pos_offset: torch.Tensor,
             block_tables: torch.Tensor, caches) -> None:
    """Move the cache rows of accepted paths together: of each sequence the row at position pos_offset +
    path[i] goes to pos_offset + i, for i < n_kept, in every layer's (k_cache, v_cache, k_scale, v_scale) of
    `caches` (all of one shape and strides, at most MAX_LAYERS), under the scales that an append of these rows
    would give their pages.  n_kept [n] and path [T] as verify_tree returns them; pos_offset [n] int32:
    the position of each sequence's token 0 (the context then is pos_offset + n_kept)."""
    caches = tuple(caches)
    if not caches:
        raise ValueError("caches is empty")
    dev = _same_device(n_kept, path, cu_seqlens, pos_offset, block_tables, *(t for layer in caches for t in layer))
    pp, T = _i32(path, "path"), path.numel()
    cu = _i32(cu_seqlens, "cu_seqlens")
    n = cu_seqlens.numel() - 1
    kp, off = _i32(n_kept, "n_kept", n), _i32(pos_offset, "pos_offset", n)
    shape, stride = caches[0][0].shape, caches[0][0].stride()
    if len(shape) != 4:
        raise ValueError("k_cache must be [num_blocks, block_size, n_kv_heads, head_dim]")
    flat, rest = [], None
    for k_cache, v_cache, k_scale, v_scale in caches:
        if k_cache.shape != shape or k_cache.stride() != stride:
            raise ValueError("the layers' caches must have one shape and the same strides")
        one = _kv8(k_cache, v_cache, k_scale, v_scale, shape[2], shape[3])
        flat += one[:4]
        rest = one[4:]
    arr = array("Q", flat)  # read by the call itself
    if _lib._recording is not None:
        _lib._held.append(arr)
    with _on_device(dev):
        _invoke(load().mrope_keep_kv8, arr.buffer_info()[0], len(caches), shape[2], shape[3], *rest, kp, pp, T, cu, n, off,
                *_tables(block_tables, n), _stream_of(dev.index))
