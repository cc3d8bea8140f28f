"""ctypes binding of the calls for trees of drafted tokens: planes and masks, attention, verification, and the
accepted path's cache rows (see include/mrope.h)."""
from __future__ import annotations

from array import array

import torch

from . import _lib
from ._kv8 import _F8, _code, _heads, _kv8, _scratch, _stream_of, _tables
from ._lib import _invoke, _on_device, load

TREE_MAX_TOKENS = 1024
MAX_LAYERS = 64
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_empty, _empty_like = torch.empty, torch.empty_like

# As in the calls of the cache: a step of few sequences spends most of its time here, so each property of a
# tensor is read once, and outputs are made like an input where one has their shape.


def _device_of(first, others) -> int:
    """Index of the one device that all tensors (None: not given) are on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("all tensors must be on a CUDA (HIP) device")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on the same CUDA (HIP) device")
    return index


def _vec(t, name: str, n: int, dtype=_I32) -> int:
    """Address of a contiguous vector of n entries."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D {str(dtype)[6:]} tensor of {n} entries")
    return t.data_ptr()


def _offsets(t):
    """(address, sequences) of cu_seqlens."""
    if t.dtype is not _I32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor")
    return t.data_ptr(), t.shape[0] - 1


def _tokens(t, name: str):
    """(address, tokens) of an int32 vector with an entry a token."""
    if t.dtype is not _I32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 tensor")
    return t.data_ptr(), t.shape[0]


def _mask(t, T: int):
    """(address, words) of a mask [tokens, words]."""
    shape = t.shape
    if t.dtype is not _I64 or len(shape) != 2 or shape[0] != T or not t.is_contiguous():
        raise ValueError("mask must be a contiguous int64 [tokens, words] tensor")
    return t.data_ptr(), shape[1]


def _call(index: int, cfunc, *args) -> None:
    """The C call, on the tensors' device and its current stream."""
    if torch._C._cuda_getDevice() == index:
        _invoke(cfunc, *args, _stream_of(index))
    else:
        with _on_device(torch.device("cuda", index)):
            _invoke(cfunc, *args, _stream_of(index))


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
    index = _device_of(parents, (cu_seqlens, pos_offset, amount, planes, mask))
    pp, T = _tokens(parents, "parents")
    cu, n = _offsets(cu_seqlens)
    off = _vec(pos_offset, "pos_offset", n)
    am = None if amount is None else _vec(amount, "amount", n)
    if planes is None:
        planes = _empty((3, T), dtype=_I32, device=parents.device)
        stride = T
    else:
        stride = planes.stride(0)
        if planes.dtype is not _I32 or planes.dim() != 2 or planes.shape[0] != 3 or planes.shape[1] < T or planes.stride(1) != 1:
            raise ValueError("planes must be an int32 [3, >= tokens] tensor with unit column stride")
    if mask is None:
        mask = _empty((T, int(mask_words)), dtype=_I64, device=parents.device)
    mp, words = _mask(mask, T)
    _call(index, load().mrope_planes_tree, pp, T, cu, n, off, am, planes.data_ptr(), stride, mp, words)
    return planes, mask


def attend_tree_kv8(q: torch.Tensor, cu_seqlens: torch.Tensor, context_lens: torch.Tensor, mask: torch.Tensor,
                    block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, *, softmax_scale: float | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None):
    """attend_kv8 under a mask over the query tokens: token i of a sequence of len sees the positions before
    context - len, and those of the sequence's tokens whose bits are set in its row of mask int64 [T, words]
    (see planes_tree).  Everything else as in attend_kv8.  Returns (out, lse or None)."""
    index = _device_of(q, (cu_seqlens, context_lens, mask, block_tables, k_cache, v_cache, k_scale, v_scale, out, lse, workspace))
    dt = _code(q)
    qp, qt, qh, nq, T, D = _heads(q, "q")
    cu, n = _offsets(cu_seqlens)
    ctx = _vec(context_lens, "context_lens", n)
    mp, words = _mask(mask, T)
    cache = _kv8(k_cache, v_cache, k_scale, v_scale, None, D)
    nk, bs, blocks = k_cache.shape[2], cache[4], cache[5]
    if out is None:
        out = _empty_like(q, memory_format=torch.contiguous_format)
        op, ot, oh = out.data_ptr(), nq * D, D
    else:
        op, ot, oh, no, _, _ = _heads(out, "out", q.dtype, T, D)
        if no != nq:
            raise ValueError("out must have q's shape")
    lp = None
    if lse is not None:
        if lse.shape != (T, nq) or lse.dtype is not _F32 or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor")
    elif return_lse:
        lse = _empty((T, nq), dtype=_F32, device=q.device)
    if lse is not None:
        lp = lse.data_ptr()
    tp, ts, tw = _tables(block_tables, n)
    lib = load()
    need = lib.mrope_attend_tree_kv8_workspace_bytes(T, n, nq, nk, D, dt, tw if blocks else 0, bs)
    ws, ws_bytes, keep = _scratch(need, q.device, workspace)
    _call(index, lib.mrope_attend_tree_kv8, qp, qt, qh, nq, T, nk, D, dt, cu, n, ctx, mp, words, tp, ts, tw, *cache,
          D ** -0.5 if softmax_scale is None else float(softmax_scale), op, ot, oh, lp, ws, ws_bytes)
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
    index = _device_of(target_probs, (ids, parents, cu_seqlens, u_accept, u_next, draft_probs, n_kept, path, next_ids, workspace))
    dt = _code(target_probs)
    ip, T = _tokens(ids, "ids")
    vocab = target_probs.shape[-1]
    tp, ts = _rows(target_probs, "target_probs", target_probs.dtype, T, vocab)
    dp, ds = (None, 0) if draft_probs is None else _rows(draft_probs, "draft_probs", target_probs.dtype, T, vocab)
    pp = None if parents is None else _vec(parents, "parents", T)
    cu, n = _offsets(cu_seqlens)
    ua, un = _vec(u_accept, "u_accept", T, _F32), _vec(u_next, "u_next", n, _F32)
    if path is None:
        path = _empty_like(ids)
    if n_kept is None:
        n_kept = _empty_like(u_next, dtype=_I32)
    if next_ids is None:
        next_ids = _empty_like(n_kept)
    lib = load()
    need = lib.mrope_verify_tree_workspace_bytes(n, vocab, dp is not None, pp is not None)
    ws, ws_bytes, keep = _scratch(need, ids.device, workspace)
    _call(index, lib.mrope_verify_tree, tp, ts, dp, ds, vocab, dt, T, ip, pp, cu, n, ua, un, _vec(n_kept, "n_kept", n),
          _vec(path, "path", T), _vec(next_ids, "next_ids", n), ws, ws_bytes)
    return n_kept, path, next_ids


def keep_kv8(n_kept: torch.Tensor, path: torch.Tensor, cu_seqlens: torch.Tensor, pos_offset: torch.Tensor,
             block_tables: torch.Tensor, caches) -> None:
    """Move the cache rows of accepted paths together: of each sequence the row at position pos_offset +
    path[i] goes to pos_offset + i, for i < n_kept, in every layer's (k_cache, v_cache, k_scale, v_scale) of
    `caches` (all of one shape and strides, at most MAX_LAYERS; a cache that layers share is given once), under
    the scales that an append of these rows would give their pages.  n_kept [n] and path [T] as verify_tree returns them; pos_offset [n] int32:
    the position of each sequence's token 0 (the context then is pos_offset + n_kept)."""
    caches = tuple(caches)
    if not caches:
        raise ValueError("caches is empty")
    layers = tuple(zip(*caches))
    if len(layers) != 4 or any(len(layer) != 4 for layer in caches):
        raise ValueError("caches must be (k_cache, v_cache, k_scale, v_scale) of each layer")
    codes, scales = layers[0] + layers[1], layers[2] + layers[3]
    index = _device_of(n_kept, (path, cu_seqlens, pos_offset, block_tables, *codes, *scales))
    pp, T = _tokens(path, "path")
    cu, n = _offsets(cu_seqlens)
    kp, off = _vec(n_kept, "n_kept", n), _vec(pos_offset, "pos_offset", n)
    k_cache = caches[0][0]
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or stride[3] != 1:
        raise ValueError("k_cache must be [num_blocks, block_size, n_kv_heads, head_dim] with contiguous head_dim")
    blocks, bs, nk, D = shape
    per_head = (blocks, nk)
    for t in codes:
        if t.shape != shape or t.stride() != stride:
            raise ValueError("the caches of all layers must have one shape and the same strides")
        if t.dtype is not _F8 and t.dtype is not torch.uint8:
            raise ValueError("caches must be float8_e4m3fn (or their codes in uint8)")
    for t in scales:
        if t.dtype is not _F32 or t.shape != per_head or not t.is_contiguous():
            raise ValueError("scales must be contiguous float32 [num_blocks, n_kv_heads] tensors")
    arr = array("Q", [t.data_ptr() for layer in caches for t in layer])  # read by the call itself
    if _lib._recording is not None:
        _lib._held.append(arr)
    _call(index, load().mrope_keep_kv8, arr.buffer_info()[0], len(caches), nk, D, bs, blocks, stride[0], stride[1], stride[2], kp, pp, T, cu,
          n, off, *_tables(block_tables, n))
