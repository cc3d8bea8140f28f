"""Cases of generating with drafted tokens over the 8-bit paged K/V cache: a tree of drafts a sequence,
attended to, verified, and its accepted path kept.

`run` computes an operator either in its plain form (elementary torch operations) or, with `own`
set, by the library's calls:

* planes   planes_tree: parents -> position planes and the mask of each drafted token's ancestors
* attend   attend_tree_kv8: attention of the drafted tokens under that mask over the cache
* verify   verify_tree: which drafted tokens the target accepts, and the token after them, from given
           random numbers
* keep     keep_kv8: the rows of the accepted path moved together in the caches of every layer
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
E_MIN, E_MAX = -96, 120  # exponents of a page scale
VOCAB = 248094           # text ids of the model that the library's rotary is for


# ---------------------------------------------------------------- cases -------------------------
def listed():
    return [
        # eight drafts for one sequence: nothing but latency
        dict(name="planes_1x8", op="planes", n=1, nodes=8, ragged=0),
        # a wide batch of trees that fill a mask word
        dict(name="planes_512x64", op="planes", n=512, nodes=64, ragged=0),
        # one sequence after a 110-token prompt, eight drafts, in fp32
        dict(name="attend_1x8_f32", op="attend", n=1, nodes=8, past=109, ragged=0, holes=False, dtype="f32", hq=8, hk=2,
             d=256, bs=16),
        # eight long sequences, sixteen drafts each: few rows, a long axis
        dict(name="attend_8x16_32k", op="attend", n=8, nodes=16, past=32000, ragged=0, holes=False, dtype="bf16", hq=8,
             hk=2, d=256, bs=16),
        # a batch of generating sequences, thirty-two drafts each, 4,096 tokens behind each
        dict(name="attend_64x32_4k", op="attend", n=64, nodes=32, past=4096, ragged=0, holes=False, dtype="bf16", hq=8,
             hk=2, d=256, bs=16),
        # trees of odd sizes, some of one token or none, fp16, narrower heads, rows that see nothing
        dict(name="attend_ragged_f16", op="attend", n=24, nodes=61, past=3001, ragged=3, holes=True, dtype="f16", hq=16,
             hk=4, d=128, bs=64),
        # wide trees of three sequences: more products than bytes
        dict(name="attend_3x250_2k", op="attend", n=3, nodes=250, past=2047, ragged=0, holes=False, dtype="bf16", hq=8,
             hk=2, d=256, bs=16),
        # one sequence, a chain of five drafts that were drawn
        dict(name="verify_chain_1x6", op="verify", n=1, nodes=6, branch=1, drawn=True, vocab=VOCAB, ragged=0, dtype="f32"),
        # trees of the drafter's best tokens, for the widest batch that keeps every distribution
        dict(name="verify_best_64x32", op="verify", n=64, nodes=32, branch=4, drawn=False, vocab=VOCAB, ragged=0,
             dtype="bf16"),
        # trees of drawn tokens: a refused sibling changes what the next one is held to
        dict(name="verify_drawn_16x13", op="verify", n=16, nodes=13, branch=3, drawn=True, vocab=VOCAB, ragged=5,
             dtype="f32"),
        # the accepted paths of eight sequences, six layers
        dict(name="keep_8x16", op="keep", n=8, nodes=16, past=333, ragged=7, layers=6, hk=2, d=256, bs=16),
        # and of a wide batch
        dict(name="keep_256x32", op="keep", n=256, nodes=32, past=90, ragged=9, layers=6, hk=2, d=256, bs=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(hi, lo))))))


def draw(rng):
    op = rng.choice(["planes", "attend", "attend", "attend", "verify", "verify", "keep"])
    ragged = rng.choice([0, rng.randrange(1, 1000)])
    hq, hk = rng.choice([(8, 2), (8, 2), (4, 4), (16, 4), (16, 2), (6, 3)])
    d, bs = rng.choice([64, 128, 256, 256]), rng.choice([16, 16, 32, 64])
    if op == "planes":
        n = _log(rng, 1, 512)
        return dict(op=op, n=n, nodes=_log(rng, 1, min(1024, 32768 // n)), ragged=rng.randrange(1, 1000))
    if op == "attend":
        nodes = _log(rng, 1, 250)
        n = _log(rng, 1, min(64, 2048 // nodes))
        # at most the products of the largest listed case, and 200,000 positions in all
        most = min(64 * 32 * 4128 * 8 * 256 // (n * nodes * hq * d) - nodes, 200000 // n, 32000)
        return dict(op=op, n=n, nodes=nodes, past=_log(rng, 1, max(1, most)), ragged=ragged, holes=rng.random() < 0.25,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), hq=hq, hk=hk, d=d, bs=bs)
    if op == "verify":
        drawn = rng.random() < 0.6
        nodes = _log(rng, 1, 13 if drawn else 32)
        vocab = rng.choice([VOCAB, _log(rng, 1000, 248094)])
        return dict(op=op, n=_log(rng, 1, (200 if drawn else 2000) // nodes), nodes=nodes, branch=rng.choice([1, 2, 3, 4]),
                    drawn=drawn, vocab=vocab, ragged=ragged, dtype=rng.choice(["bf16", "f16", "f32"]))
    n = _log(rng, 1, 256)
    return dict(op=op, n=n, nodes=_log(rng, 1, 64), past=_log(rng, 1, min(700, 25000 // n)), ragged=rng.randrange(1, 1000),
                layers=rng.choice([1, 2, 6]), hk=hk, d=d, bs=bs)


def _shape(case):
    """(drafted tokens, positions before them) of each sequence, from the case alone."""
    n, nodes, past = case["n"], case["nodes"], case.get("past", 0)
    if not case["ragged"]:
        return [nodes] * n, [past] * n
    r = random.Random(case["ragged"])
    t = [r.choice([0, 1, r.randrange(1, nodes + 1), r.randrange(max(1, nodes // 2), nodes + 1)]) for _ in range(n)]
    if not any(t):
        t[0] = nodes
    return t, [r.randrange(0, past + 1) if past else 0 for _ in range(n)]


def work(case):
    t, past = _shape(case)
    T = sum(t)
    if case["op"] == "planes":
        return {"bytes": T * (4 + 12 + 8 * _words(case)), "flops": 0}
    if case["op"] == "attend":
        es = 4 if case["dtype"] == "f32" else 2
        hq, hk, d = case["hq"], case["hk"], case["d"]
        ctx = sum(a + b for a, b in zip(t, past) if a)
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(t, past))  # (about as many drafts as a chain sees)
        return {"bytes": ctx * hk * d * 2 + T * (hq * (2 * d * es + 4) + 8 * _words(case)), "flops": 4 * pairs * hq * d}
    if case["op"] == "verify":
        es = 4 if case["dtype"] == "f32" else 2
        rows = sum(1 for a in t if a)  # where a sequence's walk ends: that row is read whole
        return {"bytes": rows * case["vocab"] * es * (2 if case["drawn"] else 1) + T * 16, "flops": 0}
    kept = sum((a + 2) // 4 for a in t)
    return {"bytes": 2 * kept * case["layers"] * case["hk"] * case["d"] * 2 + 4 * T, "flops": 0}


def _words(case):
    return -(-case["nodes"] // 64)


# ---------------------------------------------------------------- inputs ------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _running(xs):
    t = 0
    for x in xs:
        t += x
        yield t


def _tables(t, past, bs, g):
    """Pages of each sequence, in a random order over a pool with a few pages to spare."""
    need = [-(-(a + b) // bs) for a, b in zip(t, past)]
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
    s = torch.exp2(_need_exp(x.abs().amax((1, 3))).float())
    return (x / s[:, None, :, None]).to(F8), s


def _packed(t):
    """(sequence, index in it) of every token."""
    lens = torch.tensor(t, device="cuda")
    s = torch.repeat_interleave(torch.arange(len(t), device="cuda"), lens)
    return s, torch.arange(s.numel(), device="cuda") - (torch.cumsum(lens, 0) - lens)[s]


def prepare(case, seed):
    g = _gen(seed)
    t, past = _shape(case)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(case)
    st["cu"] = torch.tensor([0] + list(_running(t)), **i32)
    st["past"] = torch.tensor(past, **i32)
    st["max_t"], st["words"] = max(t), _words(case)
    T = sum(t)
    s, i = _packed(t)
    if case["op"] == "verify":
        st["parents"] = None if case["branch"] == 1 else torch.where(i > 0, (i - 1) // case["branch"], -1).int()
        return _prepare_verify(st, T, s, i, g)
    if case["op"] == "keep":
        return _prepare_keep(st, t, past, g)
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    st["parents"] = torch.where(i > 0, (u * i).long(), -1).int()  # any earlier token: a random recursive tree
    if case["op"] == "planes":
        st["past"] = torch.randint(0, 32000, (case["n"],), generator=g, **i32)
        st["amount"] = 58 * torch.randint(0, 2, (case["n"],), generator=g, **i32)
        return st
    hq, hk, d, bs = case["hq"], case["hk"], case["d"], case["bs"]
    st["mask"] = _plain_planes(dict(st, amount=st["past"]))["mask"]
    if case["holes"]:
        st["mask"] &= torch.randint(-2 ** 63, 2 ** 63 - 1, st["mask"].shape, generator=g, device="cuda")
    st["tables"], pool = _tables(t, past, bs, g)
    st["kc"], st["ks"] = _fill_cache(pool, bs, hk, d, g)
    st["vc"], st["vs"] = _fill_cache(pool, bs, hk, d, g)
    st["q"] = torch.randn(T, hq, d, generator=g, device="cuda").mul_(1.5).to(DT[case["dtype"]])
    st["ctx"] = st["past"] + torch.tensor(t, **i32)
    st["max_ctx"] = max(a + b for a, b in zip(t, past))
    return st


def _prepare_verify(st, T, s, i, g):
    """Target distributions that a few tokens of a row dominate, and drafts from a drafter that is near."""
    v, b, dt = st["vocab"], st["branch"], DT[st["dtype"]]
    logits = torch.randn(T, v, generator=g, device="cuda").mul_(2.0)
    fav = torch.arange(6, device="cuda") * (v // 6) + torch.randint(0, v // 6, (T, 6), generator=g, device="cuda")
    logits.scatter_(1, fav, 9.0 + 4.0 * torch.rand(T, 6, generator=g, device="cuda"))
    parent = (torch.where(i > 0, (i - 1) // b, 0) + st["cu"][s].long())
    which = torch.where(i > 0, (i - 1) % b, 0)
    if st["drawn"]:
        near = torch.randn(T, 6, generator=g, device="cuda").mul_(0.7)
        q = torch.softmax(logits.scatter_add(1, fav, near), 1).to(dt)
        st["draft"] = q
        at = torch.rand(T, b, generator=g, device="cuda", dtype=torch.float64)
        ids = torch.empty(T, b, dtype=torch.long, device="cuda")
        for r in range(0, T, 64):  # a child is drawn from its parent's row
            c = torch.cumsum(q[r:r + 64].double(), 1)
            ids[r:r + 64] = torch.searchsorted(c, at[r:r + 64] * c[:, -1:], right=True).clamp(max=v - 1)
        st["ids"] = ids[parent, which].int()
    else:
        st["draft"] = None
        st["ids"] = fav[parent, (which + parent) % 6].int()
    st["target"] = torch.softmax(logits, 1).to(dt)
    st["u"] = torch.rand(T, generator=g, device="cuda")
    st["u_next"] = torch.rand(st["n"], generator=g, device="cuda")
    return st


def _prepare_keep(st, t, past, g):
    """A path of each tree: its first token, then tokens one to four further."""
    n, L = st["n"], st["max_t"]
    lens = torch.tensor(t, device="cuda")
    at = torch.cumsum(torch.randint(1, 5, (n, L), generator=g, device="cuda"), 1)
    at = torch.cat([at.new_zeros(n, 1), at], 1)[:, :L]
    ends = (torch.rand(n, generator=g, device="cuda") * (at < lens[:, None]).sum(1)).long()
    on = (at < lens[:, None]) & (torch.arange(L, device="cuda") <= ends[:, None])
    st["n_kept"] = on.sum(1).int()
    s, i = _packed(t)
    st["path"] = torch.where(on, at, -1)[s, i].int()
    st["tables"], pool = _tables(t, past, st["bs"], g)
    st["caches"] = []
    for _ in range(st["layers"]):
        kc, ks = _fill_cache(pool, st["bs"], st["hk"], st["d"], g)
        vc, vs = _fill_cache(pool, st["bs"], st["hk"], st["d"], g)
        st["caches"].append((kc, vc, ks, vs))
    return st


# ---------------------------------------------------------------- one pass ----------------------
def run(st):
    if own:
        import canvas_rope_rotary_amd as mr

        if st["op"] == "planes":
            planes, mask = mr.planes_tree(st["parents"], st["cu"], st["past"], st["amount"], mask_words=st["words"])
            return {"planes": planes, "mask": mask}
        if st["op"] == "attend":
            out, lse = mr.attend_tree_kv8(st["q"], st["cu"], st["ctx"], st["mask"], st["tables"], st["kc"], st["vc"], st["ks"],
                                          st["vs"], return_lse=True)
            return {"out": out, "lse": lse}
        if st["op"] == "verify":
            n_kept, path, nxt = mr.verify_tree(st["target"], st["ids"], st["parents"], st["cu"], st["u"], st["u_next"],
                                               draft_probs=st["draft"])
            return {"n_kept": n_kept, "path": path, "next": nxt}
        mr.keep_kv8(st["n_kept"], st["path"], st["cu"], st["past"], st["tables"], st["caches"])
        return {"caches": st["caches"]}
    if st["op"] == "planes":
        return _plain_planes(st)
    if st["op"] == "attend":
        return _plain_attend(st)
    if st["op"] == "verify":
        return _plain_verify(st)
    _plain_keep(st)
    return {"caches": st["caches"]}


# ---------------------------------------------------------------- plain forms: trees ------------
def _padded(st):
    """Places of tokens in [n, max_t] arrays: (place [n, L], which are tokens, sequence and index of each token)."""
    cu, L = st["cu"].long(), st["max_t"]
    T = int(st["parents"].numel() if st.get("parents") is not None else st["ids"].numel())
    j = torch.arange(L, device="cuda")
    there = j < (cu[1:] - cu[:-1])[:, None]
    tok = torch.arange(T, device="cuda")
    s = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return (cu[:-1, None] + j).clamp(max=max(T - 1, 0)), there, s, tok - cu[s]


def _ancestors(parent):
    """[n, L, L]: whether j is i or an ancestor of it, by squaring "i or its parent"."""
    n, L = parent.shape
    j = torch.arange(L, device="cuda")
    up = ((parent[:, :, None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, (L - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _plain_planes(st):
    at, there, s, i = _padded(st)
    parent = torch.where(there, st["parents"][at].long(), -1)
    anc = _ancestors(parent)[s, i]  # [T, L]
    plane = st["past"][s] + (anc.sum(1) - 1) - st["amount"][s]
    W = st["words"]
    bit = torch.arange(64, device="cuda")
    wide = torch.cat([anc, anc.new_zeros(anc.shape[0], 64 * W - anc.shape[1])], 1).view(-1, W, 64)
    return {"planes": plane.int().expand(3, -1).contiguous(), "mask": (wide.long() << bit).sum(2)}


def _need_exp(amax):
    """Smallest e with amax <= 448 * 2^e (e4m3's largest value is 448), within the scales' range."""
    f, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (f > 0.875), E_MIN).clamp(E_MIN, E_MAX)


def _plain_attend(st):
    q, bs, n, mq, mc = st["q"], st["bs"], st["n"], st["max_t"], st["max_ctx"]
    T, hq, d = q.shape
    hk = st["hk"]
    g = hq // hk
    cu, ctx = st["cu"].long(), st["ctx"].long()
    past = ctx - (cu[1:] - cu[:-1])
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
    bits = ((st["mask"][:, :, None] >> torch.arange(64, device="cuda")) & 1).bool().view(T, -1)
    j = pos - past[:, None]  # the draft at each position
    seen = torch.gather(bits[at], 2, j.clamp(0, bits.shape[1] - 1)[:, None].expand(-1, mq, -1))
    sees = inside[:, None, :] & ((j < 0)[:, None] | seen)
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
    return {"out": out, "lse": lse[sq, :, :, t - cu[sq], 0].reshape(T, hq)}


# ---------------------------------------------------------------- plain forms: verification -----
def _plain_verify(st):
    """Every token is tested as if the walk came to it: its parent's row, less what its earlier siblings
    took.  Sums in 64 bits."""
    ids, p, draft = st["ids"].long(), st["target"], st["draft"]
    at, there, s, i = _padded(st)
    L = st["max_t"]
    j = torch.arange(L, device="cuda")
    parent = torch.where(there, j - 1, -1) if st["parents"] is None else torch.where(there, st["parents"][at].long(), -1)
    child = there & (parent >= 0)
    row = torch.gather(at, 1, parent.clamp(min=0))       # the parent's row of p
    x = ids[at]
    u = st["u"][at].double()
    px = torch.where(child, p[row, x].double(), 0.0)
    elder = child[:, :, None] & (parent[:, :, None] == parent[:, None, :]) & (j < j[:, None])  # [n, i, j]: j before i
    taken = torch.zeros(p.shape[0], dtype=torch.float64, device="cuda")
    if draft is None:
        again = (elder & (x[:, :, None] == x[:, None, :])).any(2)
        r = torch.where(again, 0.0, px)
        left = (1.0 - torch.where(elder, r[:, None, :], 0.0).sum(2)).clamp(min=0.0)
        ok = child & (u * left < r)
    else:
        qx = torch.where(child, draft[row, x].double(), 0.0)
        order = elder.sum(2)  # how many siblings come before
        z = torch.ones(p.shape[0], dtype=torch.float64, device="cuda")
        ok = torch.zeros_like(child)
        for k in range(int(st["branch"])):
            r = (px - taken[row] * qx).clamp(min=0.0)
            ok |= child & (order == k) & (u * qx * z[row] < r)
            more = torch.zeros(p.shape[0], dtype=torch.bool, device="cuda")
            more[row[child & (order == k)]] = True
            taken = torch.where(more, taken + z, taken)
            if k + 1 < int(st["branch"]):
                z = torch.where(more, _rest(p, draft, taken).sum(1), z)
    first = ok & ~(elder & ok[:, None, :]).any(2)
    first = first | (there & (j == 0))
    anc = _ancestors(parent)
    on = there & ((anc & ~first[:, None, :]).sum(2) == 0)
    n_kept = on.sum(1)
    last = torch.where(on, j, -1).amax(1)
    place = torch.where(on, torch.cumsum(on.long(), 1) - 1, L)
    path = torch.full((on.shape[0], L + 1), -1, dtype=torch.long, device="cuda")
    path.scatter_(1, place, j.expand_as(place))
    path[:, L] = -1
    # what is left where each walk ends, and the token drawn from it
    end = torch.gather(at, 1, last.clamp(min=0)[:, None])[:, 0]
    r = p[end].double()
    if draft is None:
        gone = child & (parent == last[:, None])
        mine = torch.where(gone, x, p.shape[1])
        r = torch.cat([r, r.new_zeros(r.shape[0], 1)], 1).scatter(1, mine, 0.0)[:, :-1]
    else:
        r = (r - taken[end][:, None] * draft[end].double()).clamp(min=0.0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p[end].double())
    c = torch.cumsum(r, 1)
    nxt = (c <= st["u_next"].double()[:, None] * c[:, -1:]).sum(1)
    nxt = torch.where(last >= 0, nxt.clamp(max=p.shape[1] - 1), -1)
    return {"n_kept": n_kept.int(), "path": path[s, i].int(), "next": nxt.int()}


def _rest(p, q, taken):
    """max(p - taken q, 0) of every row, in 64 bits."""
    return q.double().mul_(taken[:, None]).neg_().add_(p).clamp_(min=0.0)


# ---------------------------------------------------------------- plain forms: keep -------------
def _plain_keep(st):
    cu, bs = st["cu"].long(), st["bs"]
    T = st["path"].numel()
    tok = torch.arange(T, device="cuda")
    s = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    kept = torch.nonzero(tok - cu[s] < st["n_kept"][s])[:, 0]
    s, i = s[kept], (tok - cu[s])[kept]
    past = st["past"].long()
    of, to = past[s] + st["path"][kept].long(), past[s] + i
    tab = st["tables"].long()
    of_page, page, of_row, row = tab[s, of // bs], tab[s, to // bs], of % bs, to % bs
    # the sequences that continue inside a page, that page, and the rows it already holds
    who = torch.nonzero((past % bs > 0) & (st["n_kept"] > 0))[:, 0]
    cont = tab[who, past[who] // bs]
    rows = (torch.arange(bs, device="cuda") < (past % bs)[who, None])[:, :, None, None]
    for kc, vc, ks, vs in st["caches"]:
        for cache, scale in ((kc, ks), (vc, vs)):
            raw, hk = cache.view(torch.uint8), cache.shape[2]
            x = cache[of_page, of_row].float() * scale[of_page][:, :, None]
            amax = torch.zeros(cache.shape[0], hk, device="cuda")
            amax.scatter_reduce_(0, page[:, None].expand(-1, hk), x.abs().amax(2), "amax")
            e = _need_exp(amax)
            e_old = torch.frexp(scale[cont])[1] - 1
            e[cont] = torch.maximum(e[cont], e_old)
            now = cache[cont].float() * torch.exp2((e_old - e[cont]).float())[:, None, :, None]
            raw[cont] = torch.where(rows, now.to(F8).view(torch.uint8), raw[cont])
            raw[page, row] = (x * torch.exp2(-e[page].float())[:, :, None]).to(F8).view(torch.uint8)
            scale[page] = torch.exp2(e[page].float())


# ---------------------------------------------------------------- 64 bits -----------------------
def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits; whole numbers are not computed here."""
    if case["op"] in ("planes", "verify"):
        return None
    st = prepare(case, seed)
    return _exact_attend(st) if case["op"] == "attend" else _exact_keep(st)


def _exact_attend(st):
    bs, hk = st["bs"], st["hk"]
    T, hq, d = st["q"].shape
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    cu, ctx = st["cu"].tolist(), st["ctx"].tolist()
    words = [[w & (2 ** 64 - 1) for w in r] for r in st["mask"].tolist()]
    for s in range(st["n"]):
        lo, hi, c = cu[s], cu[s + 1], ctx[s]
        if hi == lo:
            continue
        past = c - (hi - lo)
        sees = torch.tensor([[True] * past + [words[t][j // 64] >> (j % 64) & 1 == 1 for j in range(hi - lo)]
                             for t in range(lo, hi)], device="cuda")
        pages = st["tables"][s, :-(-c // bs)].long()
        k, v = ((x[pages].double() * y[pages].double()[:, None, :, None]).reshape(-1, hk, d)[:c]
                for x, y in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        some = sees.any(1)
        for h in range(hq):
            w = st["q"][lo:hi, h].double() @ k[:, h * hk // hq].T.contiguous() / math.sqrt(d)
            w = torch.where(sees, w, -math.inf)
            z = torch.logsumexp(w, 1)
            p = torch.where(some[:, None], torch.exp(w - torch.where(some, z, 0.0)[:, None]), 0.0)
            out[lo:hi, h] = p @ v[:, h * hk // hq].contiguous()
            lse[lo:hi, h] = z
    return {"out": out, "lse": lse}


def _exact_keep(st):
    bs = st["bs"]
    cu, past, kept = st["cu"].tolist(), st["past"].tolist(), st["n_kept"].tolist()
    path, tables = st["path"].tolist(), st["tables"].tolist()
    touched = []  # (page, rows it holds, [(page, row) of the rows that come after them])
    for s in range(st["n"]):
        i = 0
        while i < kept[s]:
            p = past[s] + i
            m = min(kept[s] - i, bs - p % bs)
            src = [past[s] + path[cu[s] + i + k] for k in range(m)]
            touched.append((tables[s][p // bs], p % bs, [(tables[s][x // bs], x % bs) for x in src]))
            i += m
    got = []
    page = torch.tensor([x[0] for x in touched], dtype=torch.long, device="cuda")
    held = torch.tensor([x[1] for x in touched], dtype=torch.long, device="cuda")
    fill = [[(0, 0)] * h + src + [(0, 0)] * (bs - h - len(src)) for _, h, src in touched]
    src = torch.tensor(fill, dtype=torch.long, device="cuda").view(-1, bs, 2)
    new = torch.tensor([[h <= r < h + len(x) for r in range(bs)] for _, h, x in touched], device="cuda").view(-1, bs)
    old = torch.arange(bs, device="cuda") < held[:, None]
    for layer in st["caches"]:
        done = {}
        for c in (0, 1):
            cache, scale = layer[c].double(), layer[2 + c].double()
            x = cache[src[:, :, 0], src[:, :, 1]] * scale[src[:, :, 0]][:, :, :, None]
            x = torch.where(new[:, :, None, None], x, 0.0)
            top = x.abs().amax((1, 3))
            sc = torch.exp2(torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** E_MIN))))
            was = scale[page]
            sc = torch.where((held > 0)[:, None], torch.maximum(sc, was), sc)
            cache[page] = torch.where(old[:, :, None, None], cache[page] * (was / sc)[:, None, :, None],
                                      torch.where(new[:, :, None, None], x / sc[:, None, :, None], cache[page]))
            scale[page] = sc
            done[c], done[2 + c] = cache, scale
        got.append((done[0], done[1], done[2], done[3]))
    return {"caches": got}
