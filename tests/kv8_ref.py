"""Plain implementations, in 64 bits and on the CPU, of the 8-bit cache's append and attention and of the
page calls: loops over sequences, pages and rows, straight from the definitions in include/mrope.h."""
from __future__ import annotations

import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn
E_MIN, E_MAX = -96, 120


def rotate(x: torch.Tensor, planes: torch.Tensor, theta: float = 1e7) -> torch.Tensor:
    """x [T, h, D] (any type) -> fp32 values: pairs (j, j + 32) turned by the fp32 angle, in double,
    rounded once to fp32."""
    y = x.double().clone()
    for j in range(32):
        inv = np.float32(1.0) / np.float32(theta ** (2.0 * j / 64))
        sel = 1 if j % 3 == 1 else 2 if j % 3 == 2 and j < 30 else 0
        a = torch.from_numpy(planes[sel].numpy().astype(np.float32) * inv).double()[:, None]
        u, w = x[..., j].double(), x[..., j + 32].double()
        y[..., j] = u * a.cos() - w * a.sin()
        y[..., j + 32] = w * a.cos() + u * a.sin()
    return y.float()


def scale_exp(amax: float) -> int:
    """Smallest e >= -96 with amax <= 448 * 2^e."""
    e = E_MIN
    if amax > 0:
        e = max(E_MIN, math.ceil(math.log2(amax / 448.0)) - 2)
        while amax > 448.0 * 2.0 ** e:
            e += 1
    return min(e, E_MAX)


def append(x: torch.Tensor, cache: torch.Tensor, scale: torch.Tensor, table, pos0: int) -> None:
    """x [n, h, D] fp32 values at positions pos0.. of the sequence whose pages are `table`; cache (e4m3)
    and scale are updated in place."""
    n, h, _ = x.shape
    bs, nb = cache.shape[1], cache.shape[0]
    raw = cache.view(torch.uint8)
    i = 0
    while i < n:
        p = pos0 + i
        m = min(n - i, bs - p % bs)
        page = int(table[p // bs]) if p // bs < len(table) else -1
        if 0 <= page < nb:
            held = p % bs
            for hh in range(h):
                rows = x[i:i + m, hh].clone()
                fin = torch.isfinite(rows)
                rows[~fin] = math.nan
                amax = float(rows[fin].abs().max()) if bool(fin.any()) else 0.0
                e = scale_exp(amax)
                if held:
                    was = int(math.log2(float(scale[page, hh])))
                    if e > was:
                        old = cache[page, :held, hh].float() * 2.0 ** max(was - e, -126)
                        raw[page, :held, hh] = old.to(F8).view(torch.uint8)
                    e = max(e, was)
                raw[page, held:held + m, hh] = (rows * 2.0 ** -e).to(F8).view(torch.uint8)
                scale[page, hh] = 2.0 ** e
        i += m


def gather(cache, scale, table, n: int):
    """Positions [0, n) of a sequence as doubles [n, h, D], and which of them have a page."""
    bs, nb = cache.shape[1], cache.shape[0]
    out = torch.zeros(n, cache.shape[2], cache.shape[3], dtype=torch.float64)
    ok = torch.zeros(n, dtype=torch.bool)
    for b in range(-(-n // bs)):
        page = int(table[b]) if b < len(table) else -1
        if 0 <= page < nb:
            m = min(bs, n - b * bs)
            out[b * bs:b * bs + m] = cache[page, :m].double() * scale[page].double()[None, :, None]
            ok[b * bs:b * bs + m] = True
    return out, ok


def attend(q, cu, ctx, tables, kc, vc, ks, vs, softmax_scale=None):
    """(out [T, h, D], lse [T, h], spread [T, h, D], amp [T, h]) in 64 bits: spread = sum_j p_j |v_j| / l,
    amp = the largest sum_d |q_d k_d| * scale of the keys a row sees -- what the tolerances scale with."""
    T, hq, D = q.shape
    hk = kc.shape[2]
    g = hq // hk
    sc = D ** -0.5 if softmax_scale is None else softmax_scale
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    spread, amp = torch.zeros_like(out), torch.zeros(T, hq, dtype=torch.float64)
    n = len(ctx)
    for s in range(n):
        lo, hi = (s, s + 1) if cu is None else (int(cu[s]), int(cu[s + 1]))
        c = min(max(int(ctx[s]), 0), len(tables[s]) * kc.shape[1])
        if hi == lo or c == 0:
            continue
        k, ok = gather(kc, ks, tables[s], c)
        v, _ = gather(vc, vs, tables[s], c)
        for i in range(hi - lo):
            see = ok & (torch.arange(c) <= int(ctx[s]) - (hi - lo) + i)
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


class Pages:
    """The page state as lists."""

    def __init__(self, n_pages: int, n_rows: int, width: int, bs: int):
        self.ref = [0] * n_pages
        self.tab = [[-1] * width for _ in range(n_rows)]
        self.len = [0] * n_rows
        self.bs, self.width = bs, width

    def _need(self, n):
        return -(-n // self.bs)

    def grow(self, rows, lens):
        return self._requests([self._grow_need(i, rows, lens) for i in range(len(rows))],
                              lambda i, pages: self._grow_one(rows[i], lens[i], pages))

    def _grow_need(self, i, rows, lens):
        r = rows[i]
        if not 0 <= r < len(self.len) or r in rows[:i] or lens[i] < 0 or self._need(lens[i]) > self.width:
            return None
        return max(0, self._need(lens[i]) - self._need(self.len[r]))

    def _grow_one(self, r, n, pages):
        has = self._need(self.len[r])
        for k, p in enumerate(pages):
            self.tab[r][has + k] = p
            self.ref[p] = 1
        self.len[r] = max(self.len[r], n)

    def _requests(self, needs, do):
        free = [p for p, c in enumerate(self.ref) if c == 0]
        at, status, plan = 0, [], []
        for i, need in enumerate(needs):
            if need is None:
                status.append(2)
            elif need and at + need > len(free):
                status.append(1)
                at += need
            else:
                status.append(0)
                plan.append((i, free[at:at + need]))
                at += need
        for i, pages in plan:
            do(i, pages)
        return status

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.len):
                for k, p in enumerate(self.tab[r]):
                    if 0 <= p < len(self.ref):
                        self.ref[p] -= 1
                    self.tab[r][k] = -1
                self.len[r] = 0

    def fork(self, src, dst, pools):
        n = len(self.len)
        lens = list(self.len)
        needs = []
        for i, (s, d) in enumerate(zip(src, dst)):
            bad = not (0 <= s < n and 0 <= d < n) or d in dst[:i] or lens[d] != 0
            needs.append(None if bad else int(lens[s] % self.bs > 0))
        tab = [list(t) for t in self.tab]

        def do(i, pages):
            s, d = src[i], dst[i]
            full = lens[s] // self.bs
            row = [-1] * self.width
            for k in range(full):
                row[k] = tab[s][k]
                self.ref[row[k]] += 1
            for p in pages:
                row[full] = p
                self.ref[p] = 1
                for x in pools:
                    x[p] = x[tab[s][full]]
            self.tab[d], self.len[d] = row, lens[s]

        return self._requests(needs, do)

    def compact(self, pools):
        live = sum(c > 0 for c in self.ref)
        holes = [p for p in range(live) if self.ref[p] == 0]
        movers = [p for p in range(live, len(self.ref)) if self.ref[p] > 0]
        to = dict(zip(movers, holes))
        for m, h in to.items():
            self.ref[h], self.ref[m] = self.ref[m], 0
            for x in pools:
                x[h] = x[m]
        self.tab = [[to.get(p, p) for p in t] for t in self.tab]
        return len(movers)
