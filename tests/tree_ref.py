"""Plain implementations, in 64 bits and on the CPU, of the calls for trees of drafted tokens: loops over sequences,
tokens and rows, straight from the definitions in include/mrope.h."""
from __future__ import annotations

import math

import numpy as np
import torch

import kv8_ref

F8 = torch.float8_e4m3fn
MOST = 1024  # tokens of a tree that have parents


def parent(parents, i):
    """The parent of token i (parents: the sequence's own; None: a chain), or -1."""
    if i >= MOST:
        return -1
    p = i - 1 if parents is None else int(parents[i])
    return p if 0 <= p < i else -1


def line(parents, i):
    """Token i and its ancestors."""
    out = []
    while i >= 0:
        out.append(i)
        i = parent(parents, i)
    return out


def planes_tree(parents, cu, pos, amount, words):
    T = len(parents)
    planes = np.full((3, T), -77, np.int32)
    mask = np.full((T, words), -77, np.int64)
    for s in range(len(cu) - 1):
        mine = parents[cu[s]:cu[s + 1]]
        for i in range(len(mine)):
            up = line(mine, i)
            planes[:, cu[s] + i] = pos[s] + len(up) - 1 - (amount[s] if amount is not None else 0)
            row = [0] * words
            for j in up:
                if j < 64 * words:
                    row[j // 64] |= 1 << (j % 64)
            mask[cu[s] + i] = np.array(row, np.uint64).view(np.int64)
    return planes, mask


def bits_of(mask_row, n):
    """The first n bits of a row of int64 words."""
    words = [int(w) & (2 ** 64 - 1) for w in mask_row]
    return [bool(words[j // 64] >> (j % 64) & 1) if j // 64 < len(words) else False for j in range(n)]


def attend_tree(q, cu, ctx, mask, tables, kc, vc, ks, vs, softmax_scale=None):
    """(out, lse, spread, amp) as kv8_ref.attend has them."""
    T, hq, D = q.shape
    hk, bs = kc.shape[2], kc.shape[1]
    g = hq // hk
    sc = D ** -0.5 if softmax_scale is None else softmax_scale
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    spread, amp = torch.zeros_like(out), torch.zeros(T, hq, dtype=torch.float64)
    for s in range(len(ctx)):
        lo, hi = int(cu[s]), int(cu[s + 1])
        c = min(max(int(ctx[s]), 0), len(tables[s]) * bs)
        if hi == lo or c == 0:
            continue
        k, ok = kv8_ref.gather(kc, ks, tables[s], c)
        v, _ = kv8_ref.gather(vc, vs, tables[s], c)
        past = int(ctx[s]) - (hi - lo)
        for i in range(hi - lo):
            bits = bits_of(mask[lo + i], hi - lo)
            see = torch.tensor([j < past or bits[j - past] for j in range(c)]) & ok
            if not bool(see.any()):
                continue
            for h in range(hq):
                qq, kk, vv = q[lo + i, h].double(), k[see, h // g], v[see, h // g]
                w = (kk * qq).sum(1) * sc
                z = torch.logsumexp(w, 0)
                p = torch.exp(w - z)
                out[lo + i, h] = (p[:, None] * vv).sum(0)
                spread[lo + i, h] = (p[:, None] * vv.abs()).sum(0)
                lse[lo + i, h] = z
                amp[lo + i, h] = float((kk * qq).abs().sum(1).max()) * abs(sc)
    return out, lse, spread, amp


def _prob(row):
    x = np.asarray(row, np.float64)
    return np.where((x > 0) & (x < np.inf), x, 0.0)


def verify_one(target, ids, parents, u_accept, u_next, draft=None):
    """One sequence: rows [len, vocab] as arrays.  Returns (path, next)."""
    if len(ids) == 0:
        return [], -1
    n, vocab = min(len(ids), MOST), target.shape[1]
    path, a = [0], 0
    while True:
        r, z, found = _prob(target[a]), 1.0, False
        q = None if draft is None else _prob(draft[a])
        for x in range(a + 1, n):
            if parent(parents, x) != a or not 0 <= ids[x] < vocab:
                continue
            if float(u_accept[x]) * (1.0 if q is None else q[ids[x]]) * z < r[ids[x]]:
                path.append(x)
                a, found = x, True
                break
            if q is None:
                z = max(z - r[ids[x]], 0.0)
                r[ids[x]] = 0.0
            else:
                r = np.maximum(r - z * q, 0.0)
                z = r.sum()
        if not found:
            break
    if not r.sum() > 0:
        r = _prob(target[a])
    if not r.sum() > 0:
        return path, -1
    hit = np.nonzero((np.cumsum(r) > float(u_next) * r.sum()) & (r > 0))[0]
    return path, int(hit[0] if len(hit) else np.nonzero(r)[0][-1])


def verify_tree(target, ids, parents, cu, u_accept, u_next, draft=None):
    """(n_kept, path, next_ids) as lists; tokens behind the last sequence have None in path."""
    n_kept, path, nxt = [], [None] * len(ids), []
    for s in range(len(cu) - 1):
        lo, hi = cu[s], cu[s + 1]
        p, x = verify_one(target[lo:hi], ids[lo:hi], None if parents is None else parents[lo:hi], u_accept[lo:hi], u_next[s],
                          None if draft is None else draft[lo:hi])
        n_kept.append(len(p))
        nxt.append(x)
        path[lo:hi] = p + [-1] * (hi - lo - len(p))
    return n_kept, path, nxt


def keep(n_kept, path, cu, pos, tables, cache, scale):
    """One cache [pages, rows, heads, D] (e4m3) with its scales, in place: the kept rows' values are taken out and
    appended as kv8_ref.append does, a page at a time."""
    bs, nb = cache.shape[1], cache.shape[0]

    def page_of(s, p):
        k = p // bs
        page = int(tables[s][k]) if k < len(tables[s]) else -1
        return page if 0 <= page < nb else -1

    for s in range(len(n_kept)):
        if pos[s] < 0:
            continue
        mine, before = [], -1
        for x in path[cu[s]:cu[s + 1]][:max(n_kept[s], 0)]:
            if not before < x < cu[s + 1] - cu[s]:
                break
            mine.append(x)
            before = x
        i = 0
        while i < len(mine):
            to = pos[s] + i
            m = min(len(mine) - i, bs - to % bs)
            page = page_of(s, to)
            rows = [(to + k, pos[s] + mine[i + k]) for k in range(m)]
            rows = [(a, b) for a, b in rows if page_of(s, b) >= 0]
            if page >= 0 and rows:
                held = to % bs
                raw = cache.view(torch.uint8)
                for h in range(cache.shape[2]):
                    x = torch.stack([cache[page_of(s, b), b % bs, h].double() * float(scale[page_of(s, b), h]) for _, b in rows])
                    fin = torch.isfinite(x)
                    top = float(x[fin].abs().max()) if bool(fin.any()) else 0.0
                    e = kv8_ref.scale_exp(top)
                    if held:
                        was = int(math.log2(float(scale[page, h])))
                        if e > was:
                            old = cache[page, :held, h].float() * 2.0 ** max(was - e, -126)
                            raw[page, :held, h] = old.to(F8).view(torch.uint8)
                        e = max(e, was)
                    for (a, _), v in zip(rows, x):
                        raw[page, a % bs, h] = (v * 2.0 ** -e).float().to(F8).view(torch.uint8)
                    scale[page, h] = 2.0 ** e
            i += m
