"""Cases of the 8-bit paged K/V cache: writing it, attending over it, and managing its pages.

`run` computes an operator either in its plain form (elementary torch operations) or, with `own`
set, by the library's calls:

* append   apply_kv8 / decode_kv8: rotate Q in place, rotate K, and write K and V into paged caches
           held in e4m3 with one power-of-two scale per page and KV head
* attend   attend_kv8: causal attention of packed query tokens over that cache
* pages    pages_grow / pages_fork / pages_free / pages_compact: page tables, reference counts and
           the copies of pages that they imply
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
ROT = 64
THETA = 1e7
E_MIN, E_MAX = -96, 120  # exponents of a page scale


# ---------------------------------------------------------------- cases -------------------------
def listed():
    return [
        # one step of generation for three sequences: nothing but latency
        dict(name="append_decode_3", op="append", decode=True, n=3, lens=0, past=109, ragged=0, dtype="bf16",
             hq=8, hk=2, d=256, bs=16),
        # one step for 4,096 sequences, the widest decode batch of the benchmark
        dict(name="append_decode_4096", op="append", decode=True, n=4096, lens=0, past=500, ragged=7, dtype="bf16",
             hq=8, hk=2, d=256, bs=16),
        # pieces of prompts of odd lengths that continue inside a page, in fp32
        dict(name="append_ragged_f32", op="append", decode=False, n=37, lens=701, past=333, ragged=5, dtype="f32",
             hq=8, hk=2, d=256, bs=32),
        # 64 image prompts of 4,096 tokens
        dict(name="append_64x4096", op="append", decode=False, n=64, lens=4096, past=0, ragged=0, dtype="bf16",
             hq=8, hk=2, d=256, bs=16),
        # one sequence generating after a 110-token prompt, in fp32
        dict(name="attend_decode_1x110_f32", op="attend", n=1, lens=1, past=109, ragged=0, dtype="f32", hq=8, hk=2,
             d=256, bs=16),
        # a batch of generating sequences with 4,096 tokens behind each
        dict(name="attend_decode_64x4096", op="attend", n=64, lens=1, past=4095, ragged=0, dtype="bf16", hq=8, hk=2,
             d=256, bs=16),
        # eight long sequences generating: few rows, a long axis
        dict(name="attend_decode_8x32768", op="attend", n=8, lens=1, past=32767, ragged=0, dtype="bf16", hq=8, hk=2,
             d=256, bs=16),
        # a 16-token piece of each of three prompts on top of a long cache
        dict(name="attend_chunk_3x16", op="attend", n=3, lens=16, past=20011, ragged=0, dtype="bf16", hq=8, hk=2,
             d=256, bs=16),
        # prompts of odd lengths, some of one token or none, some continuing, fp16, narrower heads
        dict(name="attend_ragged_f16", op="attend", n=24, lens=900, past=411, ragged=3, dtype="f16", hq=16, hk=4,
             d=128, bs=64),
        # eight whole prompts of 4,096 tokens
        dict(name="attend_prefill_8x4096", op="attend", n=8, lens=4096, past=0, ragged=0, dtype="bf16", hq=8, hk=2,
             d=256, bs=16),
        # a step's turnover in a serving loop: finished rows leave, new prompts come in, some are forked
        dict(name="pages_turnover_64", op="pages", compact=False, rows=64, blocks=2048, lens=400, bs=16, hk=2, d=256,
             layers=6, fill=3),
        # a half-empty pool is compacted before the long prompts come
        dict(name="pages_compact_16384", op="pages", compact=True, rows=128, blocks=16384, lens=3000, bs=16, hk=2,
             d=256, layers=1, fill=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "pages"])
    hq, hk = rng.choice([(8, 2), (8, 2), (4, 4), (16, 4), (16, 2), (6, 3)])
    d = rng.choice([64, 128, 256, 256])
    bs = rng.choice([16, 16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    ragged = rng.randrange(1, 1000)
    if op == "append":
        if rng.random() < 0.5:
            return dict(op=op, decode=True, n=_log(rng, 1, 4096), lens=0, past=_log(rng, 1, 900), ragged=ragged,
                        dtype=dtype, hq=hq, hk=hk, d=d, bs=bs)
        n = _log(rng, 1, 64)
        return dict(op=op, decode=False, n=n, lens=_log(rng, 5, 65536 // n), past=rng.choice([0, _log(rng, 1, 700)]),
                    ragged=ragged, dtype=dtype, hq=hq, hk=hk, d=d, bs=bs)
    if op == "attend":
        kind = rng.choice(["decode", "decode", "chunk", "prefill"])
        if kind == "decode":
            n = _log(rng, 1, 64)
            return dict(op=op, n=n, lens=1, past=_log(rng, 1, min(32767, 200000 // n)), ragged=rng.choice([0, ragged]),
                        dtype=dtype, hq=hq, hk=hk, d=d, bs=bs)
        if kind == "chunk":
            n = _log(rng, 1, 16)
            return dict(op=op, n=n, lens=rng.randrange(2, 65), past=_log(rng, 16, 100000 // n // 4), ragged=0, dtype=dtype,
                        hq=hq, hk=hk, d=d, bs=bs)
        n = _log(rng, 1, 16)
        return dict(op=op, n=n, lens=_log(rng, 33, 7000 // n), past=rng.choice([0, _log(rng, 1, 500)]),
                    ragged=rng.choice([0, ragged]), dtype=dtype, hq=hq, hk=hk, d=d, bs=bs)
    rows = _log(rng, 8, 128)
    lens = _log(rng, 20, 1500)
    return dict(op=op, compact=rng.random() < 0.5, rows=rows, blocks=(rows * (lens // bs + 2)) * 2 + rng.randrange(64), lens=lens,
                bs=bs, hk=hk, d=d, layers=rng.choice([1, 2]), fill=rng.randrange(1, 1000))


def _shape(case):
    """(query tokens, tokens already in the cache) of each sequence, from the case alone."""
    n, ln, past = case["n"], case["lens"], case["past"]
    if not case["ragged"]:
        return [1 if case.get("decode") else ln] * n, [past] * n
    r = random.Random(case["ragged"])
    dec = case.get("decode") or ln == 1
    q = [1 if dec else r.choice([0, 1, r.randrange(1, ln + 1), r.randrange(max(1, ln // 2), ln + 1)]) for _ in range(n)]
    if not any(q):
        q[0] = ln
    p = [r.randrange(0, past + 1) if past else 0 for _ in range(n)]
    return q, p


def work(case):
    if case["op"] == "pages":
        pages, moved = _page_work(case)
        page = case["bs"] * case["hk"] * case["d"] * 2 + case["hk"] * 8
        return {"bytes": 8 * pages + 2 * moved * page * case["layers"], "flops": 0}
    q, p = _shape(case)
    es = 4 if case["dtype"] == "f32" else 2
    hq, hk, d = case["hq"], case["hk"], case["d"]
    T = sum(q)
    if case["op"] == "append":
        return {"bytes": T * (2 * hq * ROT * es + 2 * hk * d * es + 2 * hk * d + 12), "flops": T * (hq + hk) * ROT * 3}
    ctx = sum(a + b for a, b in zip(q, p) if a)
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(q, p))
    return {"bytes": ctx * hk * d * 2 + T * hq * (2 * d * es + 4), "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- inputs ------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tables(q, p, bs, g):
    """Pages of each sequence, in a random order over a pool with a few pages to spare."""
    need = [-(-(a + b) // bs) for a, b in zip(q, p)]
    width = max(1, max(need))
    pool = sum(need) + 3
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    cnt = torch.tensor(need, device="cuda")
    first = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(width, device="cuda")
    at = first[:, None] + col
    return torch.where(col < cnt[:, None], perm[at.clamp(max=pool - 1)], torch.tensor(-1, dtype=torch.int32, device="cuda")).contiguous(), pool


def _fill_cache(pool, bs, hk, d, g):
    """A cache as earlier appends left it: e4m3 rows under one scale for each page and head, some
    channels larger than others."""
    gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    x = torch.randn(pool, bs, hk, d, generator=g, device="cuda") * gain
    e = _need_exp(x.abs().amax((1, 3)))
    s = torch.exp2(e.float())
    return (x / s[:, None, :, None]).to(F8), s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, g)
    q_lens, past = _shape(case)
    n, bs, hq, hk, d, dt = case["n"], case["bs"], case["hq"], case["hk"], case["d"], DT[case["dtype"]]
    T = sum(q_lens)
    st = dict(case)
    st["tables"], pool = _tables(q_lens, past, bs, g)
    st["kc"], st["ks"] = _fill_cache(pool, bs, hk, d, g)
    st["vc"], st["vs"] = _fill_cache(pool, bs, hk, d, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    st["cu"] = torch.tensor([0] + list(_running(q_lens)), **i32)
    st["past"] = torch.tensor(past, **i32)
    st["q"] = torch.randn(T, hq, d, generator=g, device="cuda").mul_(1.5).to(dt)
    if case["op"] == "append":
        gain = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
        amp = torch.exp(0.4 * torch.randn(T, 1, 1, generator=g, device="cuda"))
        st["k"] = (torch.randn(T, hk, d, generator=g, device="cuda") * gain * amp).to(dt)
        st["v"] = (torch.randn(T, hk, d, generator=g, device="cuda") * amp).to(dt)
        if case["decode"]:
            st["pos"] = st["past"]
            st["amount"] = torch.where(st["past"] >= 67, 58, 0).to(torch.int32) * torch.randint(0, 2, (n,), generator=g, **i32)
        else:
            st["planes"] = _canvas(st["cu"], st["past"], T, g)
    else:
        st["ctx"] = st["past"] + torch.tensor(q_lens, **i32)
        st["max_q"], st["max_ctx"] = max(q_lens), max(a + b for a, b in zip(q_lens, past))
    return st


def _running(xs):
    t = 0
    for x in xs:
        t += x
        yield t


def _canvas(cu, past, T, g):
    """Planes of prompts with one image each, placed at a random origin."""
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    p = (past[s] + t - cu[s]).int()
    o = torch.randint(0, 40, past.shape, generator=g, device="cuda", dtype=torch.int32)[s]
    k = p - o
    row = (k >= 1) & (k <= 64)
    th = torch.where(row, o + (k - 1) // 8, torch.where(k == 0, o - 1, torch.where(k == 65, o + 8, o)))
    tw = torch.where(row, o + (k - 1) % 8, torch.where(k == 0, o - 1, torch.where(k == 65, o + 8, o)))
    out = torch.stack([torch.where(k < 0, p, torch.where(k >= 67, p - 58, x)) for x in (o, th, tw)])
    return out.int().contiguous()


# ---------------------------------------------------------------- one pass ----------------------
def run(st):
    if st["op"] == "append":
        return _run_append(st)
    if st["op"] == "attend":
        return _run_attend(st)
    return _run_pages(st)


def _run_append(st):
    if own:
        import canvas_rope_rotary_amd as mr

        if st["decode"]:
            mr.decode_kv8(st["q"], st["k"], st["v"], st["pos"], st["amount"], st["tables"], st["kc"], st["vc"],
                          st["ks"], st["vs"])
        else:
            mr.apply_kv8(st["q"], st["k"], st["v"], st["planes"], st["cu"], st["tables"], st["kc"], st["vc"],
                         st["ks"], st["vs"], pos_offset=st["past"])
    else:
        _plain_append(st)
    return {"q": st["q"], "k_cache": st["kc"], "v_cache": st["vc"], "k_scale": st["ks"], "v_scale": st["vs"]}


def _run_attend(st):
    if own:
        import canvas_rope_rotary_amd as mr

        cu = None if st["lens"] == 1 else st["cu"]
        out, lse = mr.attend_kv8(st["q"], cu, st["ctx"], st["tables"], st["kc"], st["vc"], st["ks"], st["vs"],
                                 return_lse=True)
    else:
        out, lse = _plain_attend(st)
    return {"out": out, "lse": lse}


def _run_pages(st):
    for name in ("refcount", "tables", "lens"):  # the pool as it was before the step
        st[name].copy_(st[name + "0"])
    if own:
        import canvas_rope_rotary_amd as mr

        pool = (st["refcount"], st["tables"], st["lens"])
        if st["compact"]:
            moved = mr.pages_compact(*pool, st["pools"])
            return {"refcount": pool[0], "tables": pool[1], "lens": pool[2], "moved": moved, "pools": st["pools"]}
        mr.pages_free(*pool, st["done"])
        grown = mr.pages_grow(*pool, st["new"], st["new_lens"], st["bs"])
        forked = mr.pages_fork(*pool, st["src"], st["dst"], st["bs"], st["pools"])
        return {"refcount": pool[0], "tables": pool[1], "lens": pool[2], "grown": grown, "forked": forked,
                "pools": st["pools"]}
    if st["compact"]:
        moved = _plain_compact(st)
        return {"refcount": st["refcount"], "tables": st["tables"], "lens": st["lens"], "moved": moved, "pools": st["pools"]}
    _plain_free(st)
    grown = _plain_grow(st)
    forked = _plain_fork(st)
    return {"refcount": st["refcount"], "tables": st["tables"], "lens": st["lens"], "grown": grown, "forked": forked,
            "pools": st["pools"]}


# ---------------------------------------------------------------- plain forms: append -----------
def _need_exp(amax):
    """Smallest e with amax <= 448 * 2^e (e4m3's largest value is 448), within the scales' range."""
    f, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (f > 0.875), E_MIN).clamp(E_MIN, E_MAX)


def _inv_freq():
    p = (torch.tensor(THETA, dtype=torch.float64, device="cuda") ** (torch.arange(32, device="cuda", dtype=torch.float64) * 2 / ROT)).float()
    return 1.0 / p


def _rotate(x, planes):
    """Rotate-half of the first 64 dims by the planes [3, T]: fp32 angle, products in 64 bits, one
    rounding to fp32."""
    j = torch.arange(32, device="cuda")
    sel = torch.where(j % 3 == 1, 1, torch.where((j % 3 == 2) & (j < 30), 2, 0))
    a = (planes.float()[sel].T * _inv_freq()).double()
    c, s = torch.cos(a)[:, None, :], torch.sin(a)[:, None, :]
    lo, hi = x[..., :32].double(), x[..., 32:ROT].double()
    return torch.cat([(lo * c - hi * s).float(), (hi * c + lo * s).float(), x[..., ROT:].float()], -1)


def _plain_append(st):
    q, bs = st["q"], st["bs"]
    T = q.shape[0]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    if st["decode"]:
        s, pos = t.long(), st["pos"]
        planes = (st["pos"] - st["amount"]).expand(3, T)
    else:
        s = torch.searchsorted(st["cu"][1:].contiguous(), t, right=True)
        pos = st["past"][s] + t - st["cu"][s]
        planes = st["planes"]
    q.copy_(_rotate(q, planes).to(q.dtype))
    page = st["tables"][s, (pos // bs).long()].long()
    row = (pos % bs).long()
    # the sequences that continue inside a page, that page, and the rows it already holds
    held = st["past"] % bs
    if not st["decode"]:
        held = torch.where(st["cu"][1:] > st["cu"][:-1], held, 0)
    who = torch.nonzero(held)[:, 0]
    cont = st["tables"][who, (st["past"][who] // bs).long()].long()
    rows = (torch.arange(bs, device="cuda") < held[who, None])[:, :, None, None]
    for x, cache, scale in ((_rotate(st["k"], planes), st["kc"], st["ks"]), (st["v"].float(), st["vc"], st["vs"])):
        hk, raw = x.shape[1], cache.view(torch.uint8)
        amax = torch.zeros(cache.shape[0], hk, device="cuda")
        amax.scatter_reduce_(0, page[:, None].expand(-1, hk), x.abs().amax(2), "amax")
        e = _need_exp(amax)
        e_old = torch.frexp(scale[cont])[1] - 1
        e[cont] = torch.maximum(e[cont], e_old)
        # rows already in a continued page go to its new scale
        now = cache[cont].float() * torch.exp2((e_old - e[cont]).float())[:, None, :, None]
        raw[cont] = torch.where(rows, now.to(F8).view(torch.uint8), raw[cont])
        raw[page, row] = (x * torch.exp2(-e[page].float())[:, :, None]).to(F8).view(torch.uint8)
        scale[page] = torch.exp2(e[page].float())


# ---------------------------------------------------------------- plain forms: attend -----------
def _plain_attend(st):
    q, bs, n, mq, mc = st["q"], st["bs"], st["n"], st["max_q"], st["max_ctx"]
    T, hq, d = q.shape
    hk = st["hk"]
    g = hq // hk
    cu, ctx = st["cu"].long(), st["ctx"].long()
    ln = cu[1:] - cu[:-1]
    bt = st["tables"].clamp(min=0).long()
    pos = torch.arange(mc, device="cuda")
    inside = pos < ctx[:, None]
    kv = []
    for cache, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        x = (cache[bt].float() * scale[bt][:, :, None, :, None]).reshape(n, -1, hk, d)[:, :mc]
        kv.append(torch.where(inside[:, :, None, None], x, 0.0).transpose(1, 2).contiguous())
    i = torch.arange(mq, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=T - 1)
    qp = q[at].float().reshape(n, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * mq, d)
    s = torch.matmul(qp, kv[0].transpose(2, 3).contiguous()).mul_(d ** -0.5).view(n, hk, g, mq, mc)
    sees = inside[:, None, :] & (pos <= (ctx - ln)[:, None, None] + i[:, None])
    s.masked_fill_(~sees[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hk, g * mq, mc), kv[1]).view(n, hk, g, mq, d) / torch.where(l > 0, l, 1.0)
    lse = torch.log(l) + m
    t = torch.arange(T, device="cuda")
    sq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    out = o[sq, :, :, t - cu[sq]].reshape(T, hq, d).to(q.dtype)
    return out, lse[sq, :, :, t - cu[sq], 0].reshape(T, hq)


# ---------------------------------------------------------------- plain forms: pages ------------
def _row_pages(lens, bs):
    return (lens + bs - 1) // bs


def _page_plan(case):
    """Lengths of the rows at the start, which leave, which come and which are forked, from the
    case alone."""
    r = random.Random(case["fill"])
    rows, lens = case["rows"], case["lens"]
    have = [r.randrange(max(1, lens // 2), lens + 1) for _ in range(rows)]
    idx = list(range(rows))
    r.shuffle(idx)
    k = max(1, rows // 4)
    empty, done, src = idx[:k], idx[k:2 * k], idx[2 * k:3 * k] or idx[:1]
    dst = empty[:len(empty) // 2]
    new = [x for x in empty if x not in dst] + done[:len(done) // 2]
    for x in empty:
        have[x] = 0
    src = [src[i % len(src)] for i in range(len(dst))]
    new_lens = [r.randrange(1, lens + 1) for _ in new]
    return have, done, new, new_lens, src, dst


def _page_work(case):
    have, done, new, new_lens, src, dst = _page_plan(case)
    bs = case["bs"]
    need = [-(-x // bs) for x in have]
    if case["compact"]:
        live = [b for x, b in enumerate(need) if x not in set(done)]
        pool = case["blocks"]
        # rows that left freed pages spread over the whole pool
        return pool + 2 * sum(live), int(sum(live) * (1 - sum(live) / pool))
    touched = sum(need[x] for x in done) + sum(-(-x // bs) for x in new_lens) + sum(need[x] for x in src)
    return touched + case["blocks"], sum(1 for x in src if have[x] % bs)


def _prepare_pages(case, g):
    st = dict(case)
    have, done, new, new_lens, src, dst = _page_plan(case)
    bs, hk, d, pool = case["bs"], case["hk"], case["d"], case["blocks"]
    i32 = dict(dtype=torch.int32, device="cuda")
    need = [-(-x // bs) for x in have]
    width = -(-case["lens"] // bs) + 1
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    cnt = torch.tensor(need, device="cuda")
    first = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(width, device="cuda")
    tables = torch.where(col < cnt[:, None], perm[(first[:, None] + col).clamp(max=pool - 1)], -1).int()
    lens = torch.tensor(have, **i32)
    if case["compact"]:  # some rows have left: their pages are holes
        gone = torch.tensor(done, device="cuda")
        tables[gone] = -1
        lens[gone] = 0
    ref = torch.zeros(pool + 1, **i32)
    ref.index_add_(0, torch.where(tables >= 0, tables, pool).reshape(-1).long(), torch.ones(tables.numel(), **i32))
    st.update(refcount0=ref[:pool].clone(), tables0=tables.contiguous(), lens0=lens)
    st.update(refcount=st["refcount0"].clone(), tables=st["tables0"].clone(), lens=st["lens0"].clone())
    for name, x in (("done", done), ("new", new), ("new_lens", new_lens), ("src", src), ("dst", dst)):
        st[name] = torch.tensor(x, **i32)
    pools = []
    for _ in range(case["layers"]):
        for _ in range(2):
            pools.append(torch.randn(pool, bs, hk, d, generator=g, device="cuda").to(F8))
        for _ in range(2):
            pools.append(torch.exp2(torch.randint(-4, 4, (pool, hk), generator=g, device="cuda").float()))
    st["pools"] = pools
    return st


def _plain_free(st):
    rows = st["done"].long()
    t = st["tables"][rows].long()
    pool = st["refcount"].numel()
    ref = torch.cat([st["refcount"], st["refcount"].new_zeros(1)])
    ref.index_add_(0, torch.where(t >= 0, t, pool).reshape(-1), ref.new_full((t.numel(),), -1))
    st["refcount"].copy_(ref[:pool])
    st["tables"][rows] = -1
    st["lens"][rows] = 0


def _take(st, need):
    """The first pages free, `need` of them in all the sequences' order; which sequences get theirs."""
    free = torch.nonzero(st["refcount"] == 0)[:, 0]
    end = torch.cumsum(need, 0)
    return free, end - need, end <= free.numel()


def _plain_grow(st):
    rows, bs = st["new"].long(), st["bs"]
    has, want = _row_pages(st["lens"][rows], bs).long(), _row_pages(st["new_lens"], bs).long()
    need = (want - has).clamp(min=0)
    free, first, ok = _take(st, need)
    col = torch.arange(st["tables"].shape[1], device="cuda")
    fresh = (col >= has[:, None]) & (col < want[:, None]) & ok[:, None]
    page = free[(first[:, None] + col - has[:, None]).clamp(0, free.numel() - 1)]
    st["tables"][rows] = torch.where(fresh, page.int(), st["tables"][rows])
    st["refcount"][page[fresh]] = 1
    st["lens"][rows] = torch.where(ok, torch.maximum(st["lens"][rows], st["new_lens"]), st["lens"][rows])
    return (~ok).int()


def _plain_fork(st):
    src, dst, bs = st["src"].long(), st["dst"].long(), st["bs"]
    ln = st["lens"][src].long()
    full, part = ln // bs, (ln % bs > 0).long()
    free, first, ok = _take(st, part)
    col = torch.arange(st["tables"].shape[1], device="cuda")
    t = st["tables"][src]
    shared = (col < full[:, None]) & ok[:, None]
    st["refcount"].index_add_(0, t[shared].long(), torch.ones_like(t[shared]))
    fresh = (col == full[:, None]) & (part > 0)[:, None] & ok[:, None]
    page = free[first.clamp(max=free.numel() - 1)]
    st["tables"][dst] = torch.where(shared, t, torch.where(fresh, page[:, None].int(), -1))
    to, of = page[(part > 0) & ok], t[fresh].long()
    st["refcount"][to] = 1
    st["lens"][dst] = torch.where(ok, ln, 0).int()
    for x in st["pools"]:
        x.view(torch.uint8 if x.dtype == F8 else x.dtype)[to] = x.view(torch.uint8 if x.dtype == F8 else x.dtype)[of]
    return (~ok).int()


def _plain_compact(st):
    ref = st["refcount"]
    live = ref > 0
    count = live.sum()
    at = torch.arange(ref.numel(), device="cuda")
    hole, mover = torch.nonzero(~live & (at < count))[:, 0], torch.nonzero(live & (at >= count))[:, 0]
    to = at.int()
    to[mover] = hole.int()
    t = st["tables"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()], t))
    ref[hole] = ref[mover]
    ref[mover] = 0
    for x in st["pools"]:
        x = x.view(torch.uint8) if x.dtype == F8 else x
        x[hole] = x[mover]
    return torch.full((1,), mover.numel(), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- 64 bits -----------------------
def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits; whole numbers are not computed here."""
    if case["op"] == "pages":
        return None
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attend(st)


def _exact_turned(x, planes):
    """x [T, h, d] turned pair by pair in 64 bits; the angle is the fp32 product that defines it."""
    y = x.double().clone()
    for j in range(32):
        base = torch.tensor(THETA ** (2.0 * j / ROT), dtype=torch.float64).float()
        plane = 1 if j % 3 == 1 and j < 33 else 2 if j % 3 == 2 and j < 30 else 0
        a = (planes[plane].float() * (torch.ones((), dtype=torch.float32) / base).item()).double()[:, None]
        u, w = x[..., j].double(), x[..., j + 32].double()
        y[..., j] = u * a.cos() - w * a.sin()
        y[..., j + 32] = w * a.cos() + u * a.sin()
    return y


def _exact_append(st):
    bs, n = st["bs"], st["n"]
    cu, past = st["cu"].tolist(), st["past"].tolist()
    if st["decode"]:
        planes = (st["pos"] - st["amount"]).expand(3, n)
    else:
        planes = st["planes"]
    q = _exact_turned(st["q"], planes)
    tables = st["tables"].tolist()
    got = {"q": q}
    touched = []  # (page, first row, first token, end token) of every page written
    for s in range(n):
        a, b = cu[s], cu[s + 1]
        while a < b:
            p = past[s] + a - cu[s]
            e = min(b, a + bs - p % bs)
            touched.append((tables[s][p // bs], p % bs, a, e))
            a = e
    page = torch.tensor([x[0] for x in touched], device="cuda")
    row0 = torch.tensor([x[1] for x in touched], device="cuda")
    tok0 = torch.tensor([x[2] for x in touched], device="cuda")
    tok1 = torch.tensor([x[3] for x in touched], device="cuda")
    r = torch.arange(bs, device="cuda")
    tok = tok0[:, None] + r - row0[:, None]
    new = (r >= row0[:, None]) & (tok < tok1[:, None])
    held = r < row0[:, None]
    for name, x, cache, scale in (("k", _exact_turned(st["k"], planes), st["kc"], st["ks"]),
                                  ("v", st["v"].double(), st["vc"], st["vs"])):
        cache, scale = cache.double(), scale.double()
        rows = torch.where(new[:, :, None, None], x[tok.clamp(0, x.shape[0] - 1)], 0.0)
        top = rows.abs().amax((1, 3))
        e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** E_MIN)))
        sc = torch.exp2(e)
        was = scale[page]
        sc = torch.where((row0 > 0)[:, None], torch.maximum(sc, was), sc)
        mine = torch.where(held[:, :, None, None], cache[page] * (was / sc)[:, None, :, None],
                           torch.where(new[:, :, None, None], rows / sc[:, None, :, None], cache[page]))
        cache[page] = mine
        scale[page] = sc
        got[name + "_cache"], got[name + "_scale"] = cache, scale
    return got


def _exact_attend(st):
    bs, hk = st["bs"], st["hk"]
    T, hq, d = st["q"].shape
    g = hq // hk
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    cu, ctx = st["cu"].tolist(), st["ctx"].tolist()
    for s in range(st["n"]):
        lo, hi, c = cu[s], cu[s + 1], ctx[s]
        if hi == lo or c == 0:
            continue
        pages = st["tables"][s, :-(-c // bs)].long()
        k, v = ((x[pages].double() * y[pages].double()[:, None, :, None]).reshape(-1, hk, d)[:c]
                for x, y in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        last = torch.arange(c - (hi - lo), c, device="cuda")
        for h in range(hq):
            w = st["q"][lo:hi, h].double() @ k[:, h // g].T.contiguous() / math.sqrt(d)
            w = torch.where(torch.arange(c, device="cuda") <= last[:, None], w, -math.inf)
            z = torch.logsumexp(w, 1)
            out[lo:hi, h] = torch.exp(w - z[:, None]) @ v[:, h // g].contiguous()
            lse[lo:hi, h] = z
    return {"out": out, "lse": lse}
