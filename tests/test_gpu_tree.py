"""GPU parity of the calls for trees of drafted tokens against plain 64-bit implementations (tree_ref): planes, masks, the
verification and the kept rows exactly, the attention within tolerances derived from its documented precision."""
import math
import random

import numpy as np
import pytest
import torch

import canvas_rope_rotary_amd as mr
import kv8_ref
import tree_ref as ref
from gpu_util import TORCH_DT, say
from test_gpu_kv8 import F8, HALF_STEP, World, bits, i32, same_codes
from test_gpu_kv8_precision import within

pytestmark = pytest.mark.gpu


def running(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def random_tree(n, rng, deep=0.0):
    """Parents of n tokens: any earlier one, or with probability `deep` the one before."""
    return [-1] + [i - 1 if rng.random() < deep else rng.randrange(i) for i in range(1, n)] if n else []


# ---------------------------------------------------------------- planes and masks --------------
@pytest.mark.parametrize("words", [1, 2, 16])
def test_planes_tree(words):
    """Trees from none to past the limit, chains, stars, several roots, parents that are none."""
    say("planes", words)
    rng = random.Random(words)
    lens = [1, 0, 2, 63, 64, 65, 300, 0, 1023, 1024, 1025, 1300, 5]
    trees = [random_tree(n, rng, 0.5) for n in lens]
    trees[4] = list(range(-1, 63))              # a chain
    trees[5] = [-1] + [0] * 64                  # a star
    trees[9] = list(range(-1, 1023))            # the longest chain
    trees[6] = [rng.choice([-1, -5, i, i + 3, 2 ** 31 - 1, -2 ** 31, rng.randrange(max(i, 1))]) for i in range(300)]
    par, cu = sum(trees, []), running(lens)
    pos = [rng.randrange(0, 40000) for _ in lens]
    amount = [rng.choice([0, 58, -3]) for _ in lens]
    pad = 7
    planes = torch.full((3, cu[-1] + pad + 2), -9, dtype=torch.int32, device="cuda")
    mask = torch.full((cu[-1] + pad, words), -9, dtype=torch.int64, device="cuda")
    for am in (amount, None):
        mr.planes_tree(i32(par + [0] * pad).cuda(), i32(cu).cuda(), i32(pos).cuda(), None if am is None else i32(am).cuda(),
                       planes=planes, mask=mask)
        p, m = ref.planes_tree(par, cu, pos, am, words)
        assert np.array_equal(planes[:, :cu[-1]].cpu().numpy(), p)
        assert np.array_equal(mask[:cu[-1]].cpu().numpy(), m)
        assert bool((planes[:, cu[-1]:] == -9).all()) and bool((mask[cu[-1]:] == -9).all())
    got = mr.planes_tree(i32([-1]).cuda(), i32([0, 1]).cuda(), i32([5]).cuda(), mask_words=words)
    assert got[0].tolist() == [[5]] * 3 and got[1].tolist() == [[1] + [0] * (words - 1)]


def test_planes_tree_is_decode_for_a_single_token():
    """The plane of a tree of one token is that of mr.decode: pos - amount, and a chain's planes are a prompt's."""
    planes, mask = mr.planes_tree(i32([-1, -1, 0, 1, 2]).cuda(), i32([0, 1, 5]).cuda(), i32([100, 200]).cuda(), i32([58, 0]).cuda())
    assert planes[0].tolist() == [42, 200, 201, 202, 203]
    assert mask[:, 0].tolist() == [1, 1, 3, 7, 15]


# ---------------------------------------------------------------- attention ---------------------
def tree_masks(lens, words, rng, kind):
    """Masks of `lens` tokens as the trees have them, with holes, or any bits at all."""
    trees = [random_tree(n, rng, 0.3) for n in lens]
    _, m = ref.planes_tree(sum(trees, []), running(lens), [0] * len(lens), None, words)
    noise = np.array([rng.getrandbits(64) for _ in range(m.size)], np.uint64).view(np.int64).reshape(m.shape)
    if kind == "holes":
        m &= noise
    elif kind == "any":
        m = noise
    return torch.from_numpy(m.copy())


def check_tree(w, lens, ctx, dtype, hq, *, mask=None, words=None, kind="tree", seed=0, softmax_scale=None, q=None, scale=1.0, pad=0,
               what="", call=None):
    T, cu = sum(lens), running(lens)
    words = words or -(-max(lens) // 64)
    mask = tree_masks(lens, words, random.Random(seed), kind) if mask is None else mask
    q = w.heads(T + pad, hq, dtype, scale) if q is None else q
    out = torch.full_like(q, 7.0).cuda()
    lse = torch.full((T + pad, hq), 7.0, device="cuda")
    given = torch.cat([mask, torch.full((pad, mask.shape[1]), -1, dtype=torch.int64)])
    (call or mr.attend_tree_kv8)(q.cuda(), i32(cu).cuda(), i32(ctx).cuda(), given.cuda(), w.tables.cuda(), *w.cache(),
                                 softmax_scale=softmax_scale, out=out, lse=lse)
    torch.cuda.synchronize()
    o, z, spread, amp = ref.attend_tree(q[:T], cu, ctx, mask.tolist(), w.tables.tolist(), w.kc, w.vc, w.ks, w.vs, softmax_scale)
    got, gz = out[:T].cpu().double(), lse[:T].cpu().double()
    nan = torch.isnan(o)
    assert torch.equal(nan, torch.isnan(got)) and torch.equal(torch.isnan(z), torch.isnan(gz)), what
    clean = ~torch.isnan(z)
    keep = lambda x: torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf)
    within(keep(got), torch.where(clean, gz, -math.inf), keep(o), torch.where(clean, z, -math.inf), keep(spread), keep(amp), dtype,
           q.shape[2], max(list(ctx) + [1]), what)
    assert bool((got[torch.isneginf(z)] == 0).all()), what
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all()), what
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hq,hk,bs", [(256, 8, 2, 16), (128, 16, 4, 64), (64, 3, 3, 32), (256, 4, 4, 16), (128, 14, 2, 16), (64, 64, 1, 64)])
def test_attend_ragged_trees(dtype, D, hq, hk, bs):
    """Trees from none to 40 tokens in one call (tiles of every size over the shapes), contexts from less than the
    tree to several pages, some without a context at all."""
    say("tree ragged", dtype, D, hq, hk, bs)
    lens = [1, 0, 2, 5, 33, 40, 1, 16, 3, 0, 4]
    past = [199, 5, 0, 35, 0, 91, -1, 74, -2, 0, 63]
    ctx = [max(a + b, 0) for a, b in zip(lens, past)]
    w = World(ctx, bs, hk, D, seed=D + hq + 3)
    check_tree(w, lens, ctx, dtype, hq, pad=5, kind="tree", seed=D)
    check_tree(w, lens, ctx, dtype, hq, kind="holes", seed=hq)
    check_tree(w, lens, ctx, dtype, hq, kind="any", seed=bs)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hq,hk", [(256, 8, 2), (128, 8, 1), (64, 2, 2), (256, 1, 1)])
@pytest.mark.parametrize("n", [1, 3, 8, 17])
def test_attend_few_drafts(dtype, D, hq, hk, n):
    """From one token a sequence on: tiles of 16 and 32 rows, filled in part."""
    say("tree few", dtype, D, hq, n)
    past = [130, 0, 31, 500]
    w = World([p + n for p in past], 16, hk, D, seed=D + n)
    check_tree(w, [n] * 4, [p + n for p in past], dtype, hq, seed=n)


@pytest.mark.parametrize("dtype,D,hq,hk", [("bf16", 256, 8, 2), ("f16", 128, 4, 1), ("f32", 64, 2, 2), ("f32", 256, 2, 1)])
@pytest.mark.parametrize("words", [1, 4, 5])
def test_attend_wide_trees(dtype, D, hq, hk, words):
    """Trees of several tiles and mask words; a mask that ends before the tree does, and one that goes on after it."""
    say("tree wide", dtype, D, words)
    lens = [250, 64, 130]
    ctx = [250 + 77, 64, 130 + 5]
    w = World(ctx, 32, hk, D, seed=D + words)
    check_tree(w, lens, ctx, dtype, hq, words=words, seed=words)
    check_tree(w, lens, ctx, dtype, hq, words=words, kind="any", seed=words + 9)


@pytest.mark.parametrize("dtype,hq,hk,D", [("bf16", 8, 2, 256), ("f32", 4, 2, 128), ("f16", 2, 1, 64), ("bf16", 16, 2, 128)])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_attend_long_contexts(dtype, hq, hk, D, n):
    """A long axis cut into chunks and joined, next to a short sequence in a wide table."""
    say("tree long", dtype, n)
    ctx = [9001, 50, 4096]
    w = World(ctx, 64, hk, D, seed=11)
    check_tree(w, [n] * 3, ctx, dtype, hq, seed=n)


def test_attend_long_chunks():
    """So many KV heads and long sequences that a workgroup's chunk passes 4,096 tokens (its pages are looked up again)."""
    say("tree long chunks")
    w = World([640], 16, 64, 64, seed=19)
    lens, ctx = [2, 1, 2, 1, 1, 1, 1, 0, 3], [8900] * 7 + [70, 8889]
    w.tables = w.tables[:, :40].repeat(9, 15)
    w.tables[1] = w.tables[1].flip(0)
    mask = tree_masks(lens, 1, random.Random(3), "tree")
    cu, q = running(lens), w.heads(sum(lens), 64, "bf16")
    out, lse = mr.attend_tree_kv8(q.cuda(), i32(cu).cuda(), i32(ctx).cuda(), mask.cuda(), w.tables.cuda(), *w.cache(), return_lse=True)
    heads = [0, 31, 63]
    part = [x[:, :, heads] for x in (w.kc, w.vc)] + [x[:, heads] for x in (w.ks, w.vs)]
    o, z, spread, amp = ref.attend_tree(q[:, heads], cu, ctx, mask.tolist(), w.tables.tolist(), *part)
    within(out[:, heads].cpu().double(), lse[:, heads].cpu().double(), o, z, spread, amp, "bf16", 64, 8900, "long chunks")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_seqs,hq,hk,D", [(70, 8, 2, 64), (300, 6, 3, 128), (4300, 2, 1, 64)])
def test_attend_uneven_batch(dtype, n_seqs, hq, hk, D):
    """More sequences than lanes (and than lanes squared), contexts from none to thousands."""
    say("tree uneven", dtype, n_seqs, D)
    g = torch.Generator().manual_seed(n_seqs)
    past = torch.randint(0, 60, (n_seqs,), generator=g)
    past[torch.randint(0, n_seqs, (9,), generator=g)] = torch.randint(1500, 6000, (9,), generator=g)
    past[0], past[-1], past[n_seqs // 2] = 3001, 2500, 0
    lens = [s % 5 for s in range(n_seqs)]
    lens[0], lens[-1] = 23, 9
    ctx = [int(p) + n for p, n in zip(past, lens)]
    w = World(ctx, 16, hk, D, seed=n_seqs)
    check_tree(w, lens, ctx, dtype, hq, pad=3, seed=n_seqs)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_attend_ignores_what_is_not_seen(dtype, n):
    """NaN codes, NaN and infinite scales, and bad page numbers wherever no row looks; NaN in drafts' keys and values
    reaches the rows that see them and no others."""
    say("tree unseen", dtype, n)
    ctx = [60 + n, 37 + n, 0, 30 + n]
    w = World([128, 96, 16, 80], 16, 2, 256, seed=12, width=9)
    for s, c in enumerate(ctx):
        for b in range(9):
            page = int(w.tables[s, b])
            if page < 0:
                w.tables[s, b] = [-7, w.nb, 2 ** 31 - 1][b % 3]
                continue
            used = max(0, min(16, c - 16 * b))
            w.kc.view(torch.uint8)[page, used:] = 0x7f
            w.vc.view(torch.uint8)[page, used:] = 0xff
            if used == 0:
                w.ks[page] = math.nan
                w.vs[page] = math.inf
    for kind in ("tree", "holes"):
        check_tree(w, [n] * 4, ctx, dtype, 8, kind=kind, seed=n, what="behind the end")
    # a draft's key and another's value hold NaN
    def put(cache, s, p, h, d, code):
        cache.view(torch.uint8)[int(w.tables[s, p // 16]), p % 16, h, d] = code
    put(w.vc, 0, 60 + n // 2, 0, 5, 0x7f)
    put(w.vc, 0, 60 + n // 2, 0, 201, 0xff)
    put(w.vc, 3, 30, 1, 17, 0x7f)
    put(w.kc, 1, 37 + n - 1, 1, 9, 0x7f)
    put(w.vc, 1, 3, 0, 255, 0xff)
    for kind in ("tree", "holes"):
        check_tree(w, [n] * 4, ctx, dtype, 8, kind=kind, seed=n, what="NaN")


def test_attend_unseen_pages_of_drafts():
    """A page of drafts that no row's mask names may hold anything, its scales too."""
    w = World([96], 16, 2, 128, seed=5)
    mask = torch.zeros(64, 1, dtype=torch.int64)
    mask[:, 0] = (1 << 16) - 1
    for b in range(3, 6):
        page = int(w.tables[0, b])
        w.kc.view(torch.uint8)[page], w.vc.view(torch.uint8)[page] = 0x7f, 0xff
        w.ks[page], w.vs[page] = math.inf, math.nan
    for dtype in ("bf16", "f16", "f32"):
        check_tree(w, [64], [96], dtype, 8, mask=mask, what=dtype)


def test_attend_holes_in_tables():
    """A page of the middle that is missing is not attended to; a row with missing pages only is empty; a tree
    whose own pages are missing sees its context."""
    w = World([100, 40, 33, 64], 16, 2, 128, seed=13)
    w.tables[0, 2] = -1
    w.tables[0, 6] = -1
    w.tables[1, :] = -1
    w.tables[2, 1] = w.nb + 5
    w.tables[3, 3] = -1
    for n in (1, 4, 16, 33):
        check_tree(w, [n] * 4, [100, 40, 33, 64], "bf16", 8, seed=n, what=n)


def test_attend_contexts_past_the_table():
    """A context that is longer than its table: what the table does not hold is not there, drafts included."""
    w = World([64, 48], 16, 2, 64, seed=23, width=4)
    for ctx in ([64 + 3, 48 + 40], [2 ** 31 - 1, 70], [64, 2 ** 31 - 1]):
        check_tree(w, [5, 37], ctx, "bf16", 8, seed=ctx[0] % 97, what=ctx) if max(ctx) < 1000 else None
        out, lse = mr.attend_tree_kv8(w.heads(42, 8, "bf16").cuda(), i32([0, 5, 42]).cuda(), i32(ctx).cuda(),
                                      torch.full((42, 1), -1, dtype=torch.int64).cuda(), w.tables.cuda(), *w.cache(), return_lse=True)
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


def test_attend_scores():
    """Large scores (one key takes everything), a negative and a zero factor, zero and infinite queries."""
    w = World([200, 90], 16, 2, 256, seed=14)
    lens = [40, 33]
    check_tree(w, [3, 1], [200, 90], "bf16", 8, scale=60.0)
    check_tree(w, lens, [200, 90], "bf16", 8, scale=60.0)
    for f in (0.0, -0.05, 1.0):
        check_tree(w, lens, [200, 90], "f32", 8, softmax_scale=f)
        check_tree(w, lens, [200, 90], "f16", 8, softmax_scale=f)
    q = w.heads(73, 8, "bf16")
    q[::2] = 0
    check_tree(w, lens, [200, 90], "bf16", 8, q=q)
    q = w.heads(73, 8, "f32")
    q[5, 3] *= 1e-30
    q[50, 1] = 0
    check_tree(w, lens, [200, 90], "f32", 8, q=q)
    q[:, 0, 10] = math.inf
    q[:, 1, 3] = math.nan
    out, _ = mr.attend_tree_kv8(q.cuda(), i32([0, 40, 73]).cuda(), i32([200, 90]).cuda(), torch.full((73, 1), -1, dtype=torch.int64).cuda(),
                                w.tables.cuda(), *w.cache())
    assert bool(torch.isnan(out[:, :2]).all()) and bool(torch.isfinite(out[:, 2:]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("ke,ve", [(-96, -96), (100, 118), (-20, 119)])
def test_attend_scales_at_their_ends(dtype, ke, ve):
    """Page scales at the ends of their range, other pages of the same row at the other: sums stay finite."""
    say("tree scales", dtype, ke, ve)
    w = World([300], 16, 2, 128, seed=31)
    w.ks.fill_(2.0 ** ke)
    w.vs.fill_(2.0 ** ve)
    w.vs[::2] = 2.0 ** -96
    lens = [20]
    q = w.heads(20, 8, dtype, 2.0 ** -10 if dtype == "f16" else 1.0)
    sc = 2.0 ** (-ke - 8)
    if dtype == "f16":  # the outputs pass fp16's range at both ends: what is left is that nothing is lost to a NaN
        out, lse = mr.attend_tree_kv8(q.cuda(), i32([0, 20]).cuda(), i32([300]).cuda(), torch.full((20, 1), -1, dtype=torch.int64).cuda(),
                                      w.tables.cuda(), *w.cache(), softmax_scale=sc, return_lse=True)
        assert not bool(torch.isnan(out).any()) and bool(torch.isfinite(lse).all())
        return
    out, _ = check_tree(w, lens, [300], dtype, 8, q=q, softmax_scale=sc)
    assert bool(torch.isfinite(out).all())


def test_attend_causal_masks_are_attend_kv8():
    """Chains give the causal attention: both calls within the same bound of it."""
    w = World([500, 60, 33], 16, 2, 256, seed=41)
    lens, ctx = [21, 60, 1], [500, 60, 33]
    cu = running(lens)
    par = sum(([i - 1 for i in range(n)] for n in lens), [])
    _, mask = mr.planes_tree(i32(par).cuda(), i32(cu).cuda(), i32([0] * 3).cuda())
    for dtype in ("bf16", "f16", "f32"):
        q = w.heads(cu[-1], 8, dtype)
        want = kv8_ref.attend(q, cu, ctx, w.tables.tolist(), w.kc, w.vc, w.ks, w.vs)
        args = (i32(cu).cuda(), i32(ctx).cuda())
        for name, call, extra in (("tree", mr.attend_tree_kv8, (mask,)), ("causal", mr.attend_kv8, ())):
            out, lse = call(q.cuda(), *args, *extra, w.tables.cuda(), *w.cache(), return_lse=True)
            within(out.cpu().double(), lse.cpu().double(), *want, dtype, 256, 500, (name, dtype))


def test_attend_strided_and_workspace():
    """Q and out as views, the caller's workspace, refused workspaces."""
    w = World([700, 20], 16, 2, 128, seed=15)
    lens, ctx = [9, 4], [700, 20]
    big = w.heads(13, 24, "bf16").cuda()
    q, out = big[:, 3:11], torch.zeros(13, 16, 128, dtype=torch.bfloat16, device="cuda")[:, 4:12]
    tab, cache, mask = w.tables.cuda(), w.cache(), tree_masks(lens, 1, random.Random(1), "tree")
    n = mr.attend_tree_kv8_workspace_bytes(q, 2, tab, cache[0])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    args = (q, i32([0, 9, 13]).cuda(), i32(ctx).cuda(), mask.cuda(), tab, *cache)
    mr.attend_tree_kv8(*args, out=out, workspace=ws)
    o, _, spread, _ = ref.attend_tree(q.cpu(), [0, 9, 13], ctx, mask.tolist(), w.tables.tolist(), w.kc, w.vc, w.ks, w.vs)
    assert bool(((out.cpu().double() - o).abs() <= 2.0 ** -7 * spread + 1e-9).all())
    with pytest.raises(mr.MropeError):
        mr.attend_tree_kv8(*args, workspace=ws[:n - 256])
    with pytest.raises(mr.MropeError):
        mr.attend_tree_kv8(*args, out=q)
    for bad in (mask.cuda().int(), mask.cuda()[:12], mask.cuda().flatten(), mask):
        with pytest.raises(ValueError):
            mr.attend_tree_kv8(q, args[1], args[2], bad, tab, *cache)


# ---------------------------------------------------------------- verification ------------------
def rows(T, vocab, dtype, g, sharp=3.0):
    return torch.softmax(torch.randn(T, vocab, generator=g) * sharp, 1).to(TORCH_DT[dtype])


def check_verify(target, ids, parents, cu, ua, un, draft=None, pad=0, what="", dev=None):
    """Whole numbers, equal to the plain form's."""
    T = len(ids)
    d = lambda x: x.cuda()
    path = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    tg = dev[0] if dev else d(target)
    dr = None if draft is None else (dev[1] if dev else d(draft))
    got = mr.verify_tree(tg, d(i32(ids)), None if parents is None else d(i32(parents)), d(i32(cu)), d(ua), d(un), draft_probs=dr, path=path)
    want = ref.verify_tree(target.float().numpy(), ids, parents, cu, ua.tolist(), un.tolist(), None if draft is None else draft.float().numpy())
    assert got[0].tolist() == want[0], what
    assert [x for x in got[1].tolist()] == [77 if x is None else x for x in want[1]], what
    assert got[2].tolist() == want[2], what
    return want


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [5, 1000, 2049, 40001])
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_verify(dtype, vocab, drawn, kind):
    """Trees and chains from none to 20 tokens, drafts that are likely, unlikely, repeated or outside the vocabulary."""
    say("verify", dtype, vocab, drawn, kind)
    g = torch.Generator().manual_seed(vocab + drawn)
    rng = random.Random(vocab)
    lens = [1, 0, 2, 20, 7, 1, 12, 0, 5, 20, 20, 3]
    cu, T, pad = running(lens), sum(lens), 4
    target = rows(T + pad, vocab, dtype, g)
    draft = (0.5 * target.float() + 0.5 * rows(T + pad, vocab, "f32", g)).to(target.dtype) if drawn else None
    seen, depth = set(), 0
    for turn in range(4):
        parents = sum((random_tree(n, rng, 0.2) for n in lens), []) + [0] * pad
        like = (target if draft is None else draft).float()
        ids = [-5] * (T + pad)
        for s, n in enumerate(lens):
            for i in range(1, n):
                a = cu[s] + (i - 1 if kind == "chain" else parents[cu[s] + i])
                pick = rng.random()
                ids[cu[s] + i] = (int(like[a].argmax()) if pick < 0.5 else int(torch.multinomial(like[a], 1, generator=g)) if pick < 0.9 or drawn
                                  else rng.choice([-1, vocab, 2 ** 31 - 1, rng.randrange(vocab)]))
        ua, un = torch.rand(T + pad, generator=g), torch.rand(len(lens), generator=g)
        un[0], un[2] = 0.0, 1.0 - 2.0 ** -24
        want = check_verify(target, ids, None if kind == "chain" else parents, cu, ua, un, draft, what=(dtype, vocab, turn))
        depth = max(depth, max(want[0]))
        seen |= set(want[0])
    assert depth >= 2 and len(seen) >= 3  # (0, 1 and some that went on)


def test_verify_many_siblings():
    """A star of 60 drawn drafts that are all refused: more sums than rounds; and one of 400 that were not drawn."""
    g = torch.Generator().manual_seed(4)
    vocab = 3001
    target, draft = rows(61, vocab, "f32", g), rows(61, vocab, "f32", g)
    p, q = target[0], draft[0]
    ids = [0] + [int(x) for x in torch.multinomial(q, 400, True, generator=g) if q[x] > p[x]][:60]
    assert len(ids) == 61
    ids[47] = int((p - 60 * q).argmax())
    for stop in (0, 47):  # (the drafter all but rules that token out: q Z < r whatever the random number)
        ua = torch.full((61,), 1.0 - 2.0 ** -24)
        if stop:
            ua[stop] = 0.0
        want = check_verify(target, ids, [-1] + [0] * 60, [0, 61], ua, torch.tensor([0.37]), draft, what=stop)
        assert want[0] == [2] and want[1][1] == 47
    ids[47] = ids[46]
    want = check_verify(target, ids, [-1] + [0] * 60, [0, 61], ua, torch.tensor([0.37]), draft, what="all refused")
    assert want[0] == [1]
    target = rows(401, vocab, "f32", g, 0.5)
    order = target[0].argsort(descending=True)[:400].tolist()
    for stop in (0, 399):
        ua = torch.full((401,), 1.0 - 2.0 ** -24)
        if stop:
            ua[stop] = 0.0
        want = check_verify(target, [0] + order, [-1] + [0] * 400, [0, 401], ua, torch.tensor([0.9]), what=stop)
        assert want[0] == [2 if stop else 1]


def test_verify_deep_drawn_trees():
    """Binary trees whose walk refuses the first child of every level and takes the second: a sum a level."""
    g = torch.Generator().manual_seed(9)
    vocab, n = 500, 31
    target = rows(n, vocab, "f32", g, 1.0)
    draft = rows(n, vocab, "f32", g, 1.0)
    parents = [-1] + [(i - 1) // 2 for i in range(1, n)]
    ids = [0] * n
    for i in range(1, n):
        d, t = draft[parents[i]], target[parents[i]]
        ids[i] = int((d / t).argmax()) if i % 2 else int((t - d).argmax())
    ua = torch.tensor([0.999 if i % 2 else 0.0 for i in range(n)])
    want = check_verify(target, ids, parents, [0, n], ua, torch.tensor([0.5]), draft)
    assert want[0] == [5] and want[1][:5] == [0, 2, 6, 14, 30]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_verify_rows_anywhere(dtype):
    """Rows that begin at odd elements, one behind the other or with other strides than the drafter's."""
    g = torch.Generator().manual_seed(6)
    T, vocab = 9, 4099
    target, draft = rows(T, vocab, dtype, g), rows(T, vocab, dtype, g)
    big = torch.zeros(T * (vocab + 6) + 40, dtype=TORCH_DT[dtype], device="cuda")
    for o1, s1, o2, s2 in ((0, vocab, 1, vocab), (3, vocab + 6, 0, vocab + 1), (7, vocab + 1, 5, vocab + 5)):
        views = []
        for o, s, x in ((o1, s1, target), (o2, s2, draft)):
            v = big.clone().as_strided((T, vocab), (s, 1), o)
            v.copy_(x)
            views.append(v)
        for parents in (None, [-1, 0, 0, 0, 1, 1, 2, 4, 4]):
            ids = [0] + draft[0].float().argsort(descending=True)[:8].tolist()
            check_verify(target, ids, parents, [0, 9], torch.rand(T, generator=g), torch.tensor([0.71]), draft, what=(o1, s1), dev=views)


def test_verify_without_mass():
    """Rows of zeros, NaN, negative and infinite entries; residuals that nothing is left of; numbers outside [0, 1)."""
    vocab = 2500
    t = torch.zeros(6, vocab)
    t[0, 7] = 1.0                                  # what is left of it after its only child is nothing: token 7 again
    t[1, :] = math.nan
    t[2, 3], t[2, 4], t[2, 2000] = -1.0, math.inf, 0.25
    t[3, 5] = 1e-40
    t[4, ::2] = 1.0
    cu = [0, 2, 3, 4, 5, 6]
    # sequences: (0, draft 7 refused by u = 1), (2), (3), (4), (5: nothing at all)
    ids = [0, 7, 0, 0, 0, 0]
    ua = torch.tensor([0.0, 1.0, 0, 0, 0, 0])
    for un in ([0.5] * 5, [0.0] * 5, [1.0] * 5, [2.0] * 5, [-1.0] * 5):
        want = check_verify(t, ids, None, cu, ua, torch.tensor(un), what=un)
        assert want[2][0] == 7 and want[2][1] == 2000 and want[2][2] == 5 and want[2][4] == -1
        check_verify(t, ids, None, cu, ua, torch.tensor(un), t.clone(), what=un)
        check_verify(t, ids, [-1, 0, -1, -1, -1, -1], cu, ua, torch.tensor(un), t.clone(), what=un)
    nan = mr.verify_tree(t.cuda(), i32(ids).cuda(), None, i32(cu).cuda(), ua.cuda() * math.nan, torch.full((5,), math.nan).cuda())
    assert nan[2].tolist() == [7, 2000, 5, 2498, -1]


def test_verify_long_trees():
    """Past the tokens that a tree may have: those behind are never accepted."""
    g = torch.Generator().manual_seed(8)
    vocab = 33
    for n in (1023, 1024, 1025, 1100):
        target = rows(n, vocab, "f32", g, 0.1)
        ids = torch.randint(0, vocab, (n,), generator=g).tolist()
        want = check_verify(target, ids, None, [0, n], torch.zeros(n), torch.tensor([0.5]), what=n)
        assert want[0] == [min(n, 1024)]


def test_verify_many_sequences():
    """More sequences than workgroups that run at once, and than a grid's second dimension has room for."""
    g = torch.Generator().manual_seed(10)
    n, vocab = 70000, 9
    lens = [s % 3 for s in range(n)]
    cu = running(lens)
    target = rows(cu[-1], vocab, "f32", g)
    ids = torch.randint(0, vocab, (cu[-1],), generator=g)
    ua, un = torch.rand(cu[-1], generator=g), torch.rand(n, generator=g)
    k, path, nxt = mr.verify_tree(target.cuda(), ids.int().cuda(), None, i32(cu).cuda(), ua.cuda(), un.cuda())
    first = 69000
    c0 = cu[first]
    want = ref.verify_tree(target[c0:].numpy(), ids[c0:].tolist(), None, [c - c0 for c in cu[first:]], ua[c0:].tolist(), un[first:].tolist())
    assert k[first:].tolist() == want[0] and path[c0:].tolist() == want[1] and nxt[first:].tolist() == want[2]
    assert int(k.sum()) == int((path >= 0).sum()) and bool((k.cpu() <= torch.tensor(lens)).all())


def test_drawn_drafts_leave_the_targets_distribution():
    """The first new token of 40,000 sequences of two drawn siblings, under 50 rows of a drafter that is far off: counts
    within five standard deviations of the target's."""
    g = torch.Generator().manual_seed(12)
    n, vocab = 40000, 12
    p, q = torch.softmax(torch.randn(vocab, generator=g), 0), torch.softmax(torch.randn(vocab, generator=g) * 1.5, 0)
    target, draft = p.repeat(3 * n, 1).cuda(), q.repeat(3 * n, 1).cuda()
    ids = torch.multinomial(q, 3 * n, True, generator=g).int()
    cu = torch.arange(0, 3 * n + 1, 3, dtype=torch.int32)
    k, path, nxt = mr.verify_tree(target, ids.cuda(), i32([-1, 0, 0] * n).cuda(), cu.cuda(), torch.rand(3 * n, generator=g).cuda(),
                                  torch.rand(n, generator=g).cuda(), draft_probs=draft)
    k, path, nxt = k.cpu(), path.cpu().view(n, 3), nxt.cpu()
    first = torch.where(k > 1, ids.view(n, 3).gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], nxt)
    count = torch.bincount(first.long(), minlength=vocab).double()
    sd = (n * p.double() * (1 - p.double())).sqrt()
    assert bool(((count - n * p.double()).abs() < 5 * sd).all()), (count / n, p)


# ---------------------------------------------------------------- keep --------------------------
def check_keep(w, lens, past, kept, path, layers=1, pad=0, what="", worlds=None):
    cu = running(lens)
    worlds = worlds or [w]
    caches = [x.cache() for x in worlds]
    path = path + [3] * pad
    mr.keep_kv8(i32(kept).cuda(), i32(path).cuda(), i32(cu).cuda(), i32(past).cuda(), w.tables.cuda(), [tuple(c) for c in caches])
    torch.cuda.synchronize()
    for x, (kc, vc, ks, vs) in zip(worlds, caches):
        ref.keep(kept, path[:cu[-1]], cu, past, w.tables.tolist(), x.kc, x.ks)
        ref.keep(kept, path[:cu[-1]], cu, past, w.tables.tolist(), x.vc, x.vs)
        assert torch.equal(ks.cpu(), x.ks) and torch.equal(vs.cpu(), x.vs), what
        assert same_codes(kc, x.kc) and same_codes(vc, x.vc), what
    return caches


def random_paths(lens, rng, gap=4):
    kept, path = [], []
    for n in lens:
        mine, x = [], 0
        while x < n:
            mine.append(x)
            x += rng.randrange(1, gap + 1)
        mine = mine[:rng.randrange(0, len(mine) + 1)]
        kept.append(len(mine))
        path += mine + [-1] * (n - len(mine))
    return kept, path


@pytest.mark.parametrize("D,hk,bs", [(256, 2, 16), (256, 3, 64), (128, 4, 32), (64, 1, 16), (64, 5, 64), (128, 2, 16), (256, 1, 32), (64, 2, 32), (128, 1, 64)])
def test_keep(D, hk, bs):
    """Paths of one row to several pages, in pages continued and new, scales larger and smaller on the way."""
    say("keep", D, hk, bs)
    rng = random.Random(D + bs)
    lens = [1, 0, bs, bs + 1, 3 * bs - 1, 0, 70, 5, 2, 200]
    past = [0, 7, 0, bs - 1, 3, 0, 2 * bs + 5, bs - 2, -4, 2 * bs]
    for gap in (1, 2, 5):
        w = World([max(a + b, 1) for a, b in zip(lens, past)], bs, hk, D, seed=D + bs + gap)
        w.ks *= torch.exp2(torch.randint(-3, 4, w.ks.shape, generator=w.g).float())
        w.vs[::3] *= 2.0 ** 12
        kept, path = random_paths(lens, rng, gap)
        if gap == 1:
            kept, path = lens, sum((list(range(n)) for n in lens), [])  # everything is kept: pages may be re-coded in place
        check_keep(w, lens, past, kept, path, pad=3, what=gap)


def test_keep_layers_and_strides():
    """Six layers of views into one buffer, each its own codes and scales."""
    g = torch.Generator().manual_seed(3)
    base = World([90, 33, 70], 16, 2, 128, seed=50)
    worlds = [World([90, 33, 70], 16, 2, 128, seed=50 + i) for i in range(6)]
    big = torch.zeros(base.nb, 16, 6, 2, 2, 128, dtype=torch.uint8, device="cuda")
    caches = []
    for i, x in enumerate(worlds):
        kc, vc = big[:, :, i, 0].view(F8), big[:, :, i, 1].view(F8)
        kc.view(torch.uint8).copy_(x.kc.view(torch.uint8))
        vc.view(torch.uint8).copy_(x.vc.view(torch.uint8))
        caches.append((kc, vc, x.ks.clone().cuda(), x.vs.clone().cuda()))
    lens, past = [30, 33, 20], [60, 0, 50]
    kept, path = random_paths(lens, random.Random(5), 3)
    kept[0], path[:30] = 9, [0, 2, 5, 8, 9, 14, 20, 21, 29] + [-1] * 21
    mr.keep_kv8(i32(kept).cuda(), i32(path).cuda(), i32(running(lens)).cuda(), i32(past).cuda(), base.tables.cuda(), caches)
    for (kc, vc, ks, vs), x in zip(caches, worlds):
        ref.keep(kept, path, running(lens), past, base.tables.tolist(), x.kc, x.ks)
        ref.keep(kept, path, running(lens), past, base.tables.tolist(), x.vc, x.vs)
        assert torch.equal(ks.cpu(), x.ks) and torch.equal(vs.cpu(), x.vs)
        assert same_codes(kc.contiguous(), x.kc) and same_codes(vc.contiguous(), x.vc)
    del g


def test_keep_refuses_bad_paths_row_by_row():
    """Entries that do not ascend, lie outside the tree, or are more than there are end the list; missing pages are passed
    over; NaN codes stay NaN and have no part in a scale."""
    w = World([60, 60, 60, 60, 60, 60], 16, 2, 64, seed=61)
    w.kc.view(torch.uint8)[int(w.tables[5, 2]), 3, 0, 7] = 0x7f
    w.vc.view(torch.uint8)[int(w.tables[5, 2]), 4] = 0xff
    w.tables[3, 2] = -1                 # sources of the page are missing
    w.tables[4, 1] = w.nb + 3           # where rows would go
    lens, past = [40] * 6, [20, 20, 5, 20, 10, 20]
    lists = [[0, 3, 3, 9], [0, 5, 41, 42], [2, 1], [0, 12, 13, 14, 30], [0, 1, 2, 3, 4, 5, 6, 8, 9, 30, 31], [0, 15, 16, 17, 39]]
    kept = [4, 4, 2, 5, 11, 99]
    path = sum((x + [-1] * (40 - len(x)) for x in lists), [])
    check_keep(w, lens, past, kept, path)
    w = World([60], 16, 1, 64, seed=62)
    check_keep(w, [40], [20], [-3], list(range(40)))
    check_keep(w, [40], [20], [2 ** 31 - 1], list(range(0, 40, 2)) + [-1] * 20)
    check_keep(w, [40], [2 ** 31 - 1], [5], [0, 1, 2, 4, 9] + [-1] * 35)


def test_keep_scales_at_their_ends():
    w = World([64], 16, 2, 128, seed=63)
    w.ks.fill_(2.0 ** 120)
    w.ks[int(w.tables[0, 3])] = 2.0 ** -96
    w.vs.fill_(2.0 ** -96)
    w.vc.view(torch.uint8)[int(w.tables[0, 2])] = 0
    check_keep(w, [44], [20], [9], [0, 3, 5, 12, 14, 28, 29, 30, 43] + [-1] * 35)


# ---------------------------------------------------------------- together ----------------------
@pytest.mark.parametrize("dtype,drawn", [("bf16", False), ("f32", True), ("f16", True)])
def test_a_step_of_generation(dtype, drawn):
    """Steps as a serving loop makes them -- pages grow, planes and masks, rotary and append, attention, verification,
    keep -- each against the plain forms on the same state, which the next step goes on from."""
    say("step", dtype, drawn)
    rng, g = random.Random(17), torch.Generator().manual_seed(17)
    n, hq, hk, D, bs, vocab, layers = 3, 4, 2, 128, 16, 700, 2
    nb, width = 64, 12
    state = (torch.zeros(nb, dtype=torch.int32, device="cuda"), torch.full((n, width), -1, dtype=torch.int32, device="cuda"),
             torch.zeros(n, dtype=torch.int32, device="cuda"))
    host = [[torch.zeros(nb, bs, hk, D).to(F8), torch.zeros(nb, bs, hk, D).to(F8), torch.ones(nb, hk), torch.ones(nb, hk)] for _ in range(layers)]
    caches = [tuple(x.clone().cuda() for x in layer) for layer in host]
    past, amount = [0] * n, [0, 5, 0]
    all_rows = i32(range(n)).cuda()
    for step in range(5):
        lens = [[40, 17, 30], [9, 1, 20], [33, 12, 0], [1, 1, 1], [16, 24, 8]][step]
        cu, T = running(lens), sum(lens)
        trees = [list(range(-1, m - 1)) if step == 0 else random_tree(m, rng, 0.4) for m in lens]
        par = sum(trees, [])
        status = mr.pages_grow(*state, all_rows, i32([p + m for p, m in zip(past, lens)]).cuda(), bs)
        assert status.tolist() == [0] * n
        tables = state[1].tolist()
        cud, pos = i32(cu).cuda(), i32(past).cuda()
        planes, mask = mr.planes_tree(i32(par).cuda(), cud, pos, i32(amount).cuda())
        want_planes, want_mask = ref.planes_tree(par, cu, past, amount, 1)
        assert np.array_equal(planes.cpu().numpy(), want_planes) and np.array_equal(mask.cpu().numpy(), want_mask)
        ctx = [p + m for p, m in zip(past, lens)]
        for layer, (kc, vc, ks, vs) in zip(host, caches):
            q, k, v = (torch.randn(T, h, D, generator=g).to(TORCH_DT[dtype]) for h in (hq, hk, hk))
            qd = q.cuda()
            mr.apply_kv8(qd, k.cuda(), v.cuda(), planes, cud, state[1], kc, vc, ks, vs, pos_offset=pos)
            kr = kv8_ref.rotate(k, torch.from_numpy(want_planes))
            for s in range(n):
                kv8_ref.append(kr[cu[s]:cu[s + 1]], layer[0], layer[2], tables[s], past[s])
                kv8_ref.append(v[cu[s]:cu[s + 1]].float(), layer[1], layer[3], tables[s], past[s])
            assert same_codes(kc, layer[0]) and same_codes(vc, layer[1])
            out, lse = mr.attend_tree_kv8(qd, cud, i32(ctx).cuda(), mask, state[1], kc, vc, ks, vs, return_lse=True)
            o, z, spread, amp = ref.attend_tree(qd.cpu(), cu, ctx, want_mask.tolist(), tables, *layer)
            within(out.cpu().double(), lse.cpu().double(), o, z, spread, amp, dtype, D, 200, (step, dtype))
        target = rows(T, vocab, dtype, g)
        draft = rows(T, vocab, dtype, g) if drawn else None
        ids = [0] * T
        for s in range(n):
            for i in range(1, lens[s]):
                ids[cu[s] + i] = int(target[cu[s] + max(trees[s][i], 0)].float().argmax())
        ua, un = torch.rand(T, generator=g) * 0.5, torch.rand(n, generator=g)
        kept, path, nxt = mr.verify_tree(target.cuda(), i32(ids).cuda(), i32(par).cuda(), cud, ua.cuda(), un.cuda(),
                                         draft_probs=None if draft is None else draft.cuda())
        want = ref.verify_tree(target.float().numpy(), ids, par, cu, ua.tolist(), un.tolist(), None if draft is None else draft.float().numpy())
        assert (kept.tolist(), path.tolist(), nxt.tolist()) == tuple(want)
        mr.keep_kv8(kept, path, cud, pos, state[1], caches)
        for layer, (kc, vc, ks, vs) in zip(host, caches):
            ref.keep(want[0], want[1], cu, past, tables, layer[0], layer[2])
            ref.keep(want[0], want[1], cu, past, tables, layer[1], layer[3])
            assert same_codes(kc, layer[0]) and same_codes(vc, layer[1])
            assert torch.equal(ks.cpu(), layer[2]) and torch.equal(vs.cpu(), layer[3])
        past = [p + k for p, k in zip(past, want[0])]
    assert sum(past) > 5 * n  # some drafts were kept


def graph_world(seed=70):
    g = torch.Generator().manual_seed(seed)
    w = World([340, 90, 61], 16, 2, 256, seed=seed)
    lens, past, vocab = [24, 9, 40], [310, 70, 20], 9001
    rng = random.Random(seed)

    def inputs():
        par = sum((random_tree(m, rng, 0.4) for m in lens), [])
        T = sum(lens)
        return [i32(par).cuda(), w.heads(T, 8, "bf16").cuda(), torch.softmax(torch.randn(T, vocab, generator=g) * 4, 1).cuda(),
                torch.softmax(torch.randn(T, vocab, generator=g) * 4, 1).cuda(),
                torch.randint(0, vocab, (T,), generator=g).int().cuda(), torch.rand(T, generator=g).cuda() * 0.2, torch.rand(3, generator=g).cuda()]
    return w, lens, past, inputs


def test_graph_replay_streams_and_prepared_calls():
    """A step captured and replayed with new inputs, eager work between the replays; two graphs of the same step;
    the same calls on a side stream, two at once; prepared calls."""
    w, lens, past, inputs = graph_world()
    cu, tab = i32(running(lens)).cuda(), w.tables.cuda()
    pos, ctx = i32(past).cuda(), i32([a + b for a, b in zip(past, lens)]).cuda()
    T = sum(lens)
    cache = w.cache()
    buf = inputs()
    par, q, target, draft, ids, ua, un = buf

    def outputs():
        return [torch.empty((3, T), dtype=torch.int32, device="cuda"), torch.empty((T, 1), dtype=torch.int64, device="cuda"),
                torch.empty_like(q), torch.empty((T, 8), device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda"),
                torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")]

    outs = outputs()

    def step(o=outs, c=cache):
        mr.planes_tree(par, cu, pos, planes=o[0], mask=o[1])
        mr.attend_tree_kv8(q, cu, ctx, o[1], tab, *c, out=o[2], lse=o[3])
        mr.verify_tree(target, ids, par, cu, ua, un, draft_probs=draft, n_kept=o[4], path=o[5], next_ids=o[6])
        mr.keep_kv8(o[4], o[5], cu, pos, tab, [tuple(c)])

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        graphs.append(gr)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(6):
        new = inputs()
        state = [x.clone() for x in w.cache()]

        def put():
            for a, b in zip(buf, new):
                a.copy_(b)
            for a, b in zip(cache, state):
                a.view(torch.uint8).copy_(b.view(torch.uint8))

        put()
        step()
        want, codes = [x.clone() for x in outs], [bits(x).clone() for x in cache]
        torch.cuda.synchronize()
        put()
        for x in outs:
            x.zero_()
        if i < 4:
            graphs[i % 2].replay()
            sides = []
        else:
            sides = [(outputs(), [x.clone() for x in state]) for _ in side]
            for st, (o, c) in zip(side, sides):
                st.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(st):
                    step(o, c)
            for st in side:
                torch.cuda.current_stream().wait_stream(st)
            step()
        for o, c in [(outs, cache)] + sides:
            assert all(torch.equal(a, b) for a, b in zip(o, want)), i
            assert all(torch.equal(bits(a), b) for a, b in zip(c, codes)), i
        torch.ones(1 << 20, device="cuda").sum().item()  # eager work between the replays
    runs = [mr.prepare(mr.planes_tree, par, cu, pos, planes=outs[0], mask=outs[1]),
            mr.prepare(mr.attend_tree_kv8, q, cu, ctx, outs[1], tab, *cache, out=outs[2], lse=outs[3]),
            mr.prepare(mr.verify_tree, target, ids, par, cu, ua, un, draft_probs=draft, n_kept=outs[4], path=outs[5], next_ids=outs[6]),
            mr.prepare(mr.keep_kv8, outs[4], outs[5], cu, pos, tab, [tuple(cache)])]
    for _ in range(3):
        for a, b in zip(buf, inputs()):
            a.copy_(b)
        before = [x.clone() for x in cache]
        step()
        want, codes = [x.clone() for x in outs], [bits(x).clone() for x in cache]
        for a, b in zip(cache, before):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        for x in outs:
            x.zero_()
        junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        for run in runs:
            run()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(bits(a), b) for a, b in zip(cache, codes))
        del junk


def test_empty_batches():
    z = torch.zeros
    cu = i32([0, 0, 0]).cuda()
    none = i32([]).cuda()
    planes, mask = mr.planes_tree(none, cu, i32([1, 2]).cuda())
    assert planes.shape == (3, 0) and mask.shape == (0, 1)
    k, path, nxt = mr.verify_tree(z(0, 50, device="cuda"), none, None, cu, z(0, device="cuda"), z(2, device="cuda"))
    assert k.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and path.numel() == 0
    w = World([20, 20], 16, 2, 64, seed=1)
    cache = w.cache()
    mr.keep_kv8(k, path, cu, i32([0, 0]).cuda(), w.tables.cuda(), [tuple(cache)])
    assert same_codes(cache[0], w.kc)
    out, _ = mr.attend_tree_kv8(w.heads(0, 8, "bf16").cuda(), cu, i32([20, 20]).cuda(), mask, w.tables.cuda(), *cache)
    assert out.shape == (0, 8, 64)


def test_binding_refusals():
    w = World([20, 20], 16, 2, 128, seed=16)
    kc, vc, ks, vs = w.cache()
    tab = w.tables.cuda()
    cu, two, par = i32([0, 1, 3]).cuda(), i32([1, 2]).cuda(), i32([-1, -1, 0]).cuda()
    t, u, un = torch.rand(3, 50, device="cuda"), torch.rand(3, device="cuda"), torch.rand(2, device="cuda")
    for kw in (dict(parents=par.long()), dict(pos_offset=two[:1]), dict(amount=two.float()), dict(mask_words=0), dict(mask_words=17),
               dict(planes=torch.zeros(3, 2, dtype=torch.int32, device="cuda")), dict(mask=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises((ValueError, TypeError, mr.MropeError)):
            mr.planes_tree(**{**dict(parents=par, cu_seqlens=cu, pos_offset=two), **kw})
    ver = dict(target_probs=t, ids=par, parents=par, cu_seqlens=cu, u_accept=u, u_next=un)
    for kw in (dict(target_probs=t.double()), dict(target_probs=t[:2]), dict(target_probs=t.t()), dict(draft_probs=t.half()),
               dict(draft_probs=t[:, :49]), dict(ids=par.long()), dict(parents=par[:2]), dict(u_accept=u.double()), dict(u_next=u),
               dict(path=par[:2]), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(u_next=un.cpu())):
        with pytest.raises((ValueError, TypeError, mr.MropeError)):
            mr.verify_tree(**{**ver, **kw})
    keep = dict(n_kept=two, path=par, cu_seqlens=cu, pos_offset=two, block_tables=tab, caches=[(kc, vc, ks, vs)])
    for kw in (dict(path=par.long()), dict(n_kept=par), dict(caches=[]), dict(caches=[(kc, vc, ks, vs), (kc[1:], vc[1:], ks[1:], vs[1:])]),
               dict(caches=[(kc, vc, ks.half(), vs)]), dict(block_tables=tab[:1]), dict(caches=[(kc.float(), vc, ks, vs)]),
               dict(caches=[(kc, vc, ks, vs)] * 65), dict(caches=[(kc.cpu(), vc, ks, vs)])):
        with pytest.raises((ValueError, TypeError, mr.MropeError)):
            mr.keep_kv8(**{**keep, **kw})
