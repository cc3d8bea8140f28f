"""GPU edges of the calls for trees of drafted tokens: caches laid out otherwise, offsets past 32 bits, batches around the limits
at which a kernel cuts its work differently, the smallest and largest vocabularies."""
import random

import pytest
import torch

import canvas_rope_rotary_amd as mr
import tree_ref as ref
from gpu_util import TORCH_DT, say
from test_gpu_kv8 import F8, World, i32, same_codes
from test_gpu_kv8_precision import within
from test_gpu_tree import check_tree, random_paths, random_tree, running, tree_masks

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- attention ---------------------
def turned(w, gap):
    """The world's caches with heads before rows, and `gap` rows more a page than it has."""
    out = []
    for x in w.cache()[:2]:
        room = torch.full((w.nb, w.hk, w.bs + gap, w.D), 0x7f, dtype=torch.uint8, device="cuda")  # NaN codes around it
        y = room[:, :, :w.bs].transpose(1, 2)
        y.copy_(x.view(torch.uint8))
        out.append(y)
    return out


@pytest.mark.parametrize("dtype,D,bs", [("bf16", 256, 16), ("f16", 128, 64), ("f32", 64, 32), ("f32", 256, 16)])
def test_attend_head_major_cache(dtype, D, bs):
    say("tree head-major", dtype, D)
    lens, ctx = [40, 3, 70], [400, 90, 70]
    w = World(ctx, bs, 3, D, seed=170 + D)
    kc, vc = turned(w, 8)

    def call(q, cu, c, mask, tables, _k, _v, ks, vs, **kw):
        return mr.attend_tree_kv8(q, cu, c, mask, tables, kc, vc, ks, vs, **kw)

    check_tree(w, lens, ctx, dtype, 6, seed=D, call=call)


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("f16", 64), ("f32", 128)])
def test_attend_pool_past_two_gib(dtype, D):
    """Pages past 2^31 bytes of a pool give what the same pages of a small pool do, bit for bit."""
    say("tree large pool", dtype, D)
    w = World([600, 50], 64, 2, D, seed=171)
    small = w.cache()
    big_n = (1 << 31) // (64 * 2 * D) + 200
    move = big_n - w.nb
    big = [torch.zeros(big_n, *x.shape[1:], dtype=torch.uint8 if x.dtype == F8 else x.dtype, device="cuda") for x in small]
    for a, b in zip(big, small):
        a[move:] = b.view(a.dtype)
    far = torch.where(w.tables >= 0, w.tables + move, w.tables).cuda()
    lens = [33, 20]
    mask = tree_masks(lens, 1, random.Random(4), "tree").cuda()
    q, cu, ctx = w.heads(53, 6, dtype).cuda(), i32(running(lens)).cuda(), i32([600, 50]).cuda()
    a = mr.attend_tree_kv8(q, cu, ctx, mask, w.tables.cuda(), *small, return_lse=True)
    b = mr.attend_tree_kv8(q, cu, ctx, mask, far, *big, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("bf16", 128), ("f16", 64)])
def test_attend_rows_far_apart(dtype, D):
    """Rows of a page as far from one another as a row's stride may be (2^28 - 16 bytes): offsets up to 2^32 in a page."""
    say("tree far rows", dtype, D)
    w = World([32], 16, 1, D, seed=172, extra=0)
    stride = (1 << 28) - 16
    room = torch.empty(2, w.nb * (16 * stride // w.nb) + D, dtype=torch.uint8, device="cuda")
    caches = []
    for r, x in zip(room, w.cache()[:2]):
        y = torch.as_strided(r, (w.nb, 16, 1, D), (D, stride, D, 1))  # (two pages side by side)
        y.copy_(x.view(torch.uint8))
        caches.append(y)

    def call(q, cu, c, mask, tables, _k, _v, ks, vs, **kw):
        return mr.attend_tree_kv8(q, cu, c, mask, tables, *caches, ks, vs, **kw)

    check_tree(w, [5], [32], dtype, 4, seed=D, call=call)


@pytest.mark.parametrize("dtype,D,hq,hk", [("bf16", 256, 2, 1), ("f16", 128, 8, 2), ("bf16", 64, 4, 4), ("f32", 128, 1, 1), ("f32", 256, 2, 2)])
@pytest.mark.parametrize("n_seqs", [63, 64, 65, 127, 128, 129, 256, 257])
def test_attend_batches_around_the_limits(dtype, D, hq, hk, n_seqs):
    """As many sequences as lanes, as workgroups that run at once, and one more or less, most of them short and some long
    enough to be cut; trees of none to a few tokens."""
    say("tree limits", dtype, D, n_seqs)
    rng = random.Random(n_seqs + D)
    lens = [rng.choice([0, 1, 1, 2, 5]) for _ in range(n_seqs)]
    ctx = [a + (rng.choice([0, 3, 60]) if s % 29 else 2100) for s, a in enumerate(lens)]
    lens[0], ctx[0] = 3, 2103
    w = World(ctx, 64, hk, D, seed=n_seqs)
    check_tree(w, lens, ctx, dtype, hq, seed=n_seqs)


@pytest.mark.parametrize("dtype,D,hq,n_seqs,len0", [
    ("bf16", 256, 8, 4, 8), ("bf16", 256, 8, 5, 8), ("bf16", 256, 8, 32, 32), ("bf16", 256, 8, 33, 32), ("f16", 128, 16, 33, 16),
    ("bf16", 64, 8, 33, 40), ("f16", 256, 16, 65, 9)])
def test_attend_tiles_that_run_at_once_and_more(dtype, D, hq, n_seqs, len0):
    """Both widths of tiles, on either side of the limit between them, over contexts of unlike lengths."""
    say("tree tiles", dtype, D, n_seqs)
    lens = [len0] * n_seqs
    ctx = [len0 + (37 * s) % 300 + (1200 if s % 7 == 0 else 0) for s in range(n_seqs)]
    w = World(ctx, 16, 2, D, seed=n_seqs + D)
    check_tree(w, lens, ctx, dtype, hq, seed=len0)


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("f16", 128), ("bf16", 64), ("f32", 64), ("f32", 256)])
@pytest.mark.parametrize("n_seqs", [3, 6])
def test_attend_chunks_past_a_look_up(dtype, D, n_seqs):
    """Whole contexts of some thousand tokens a workgroup, in both widths of tiles: the pages are looked up again on the way."""
    say("tree look-ups", dtype, D, n_seqs)
    w = World([640], 16, 64, D, seed=173)
    lens, ctx = [2] * n_seqs, [8900] * (n_seqs - 1) + [8300]
    w.tables = w.tables[:, :40].repeat(n_seqs, 15)
    w.tables[1] = w.tables[1].flip(0)
    mask = tree_masks(lens, 1, random.Random(3), "tree")
    cu, q = running(lens), w.heads(sum(lens), 64, dtype)
    out, lse = mr.attend_tree_kv8(q.cuda(), i32(cu).cuda(), i32(ctx).cuda(), mask.cuda(), w.tables.cuda(), *w.cache(), return_lse=True)
    heads = [0, 63]
    part = [x[:, :, heads] for x in (w.kc, w.vc)] + [x[:, heads] for x in (w.ks, w.vs)]
    o, z, spread, amp = ref.attend_tree(q[:, heads], cu, ctx, mask.tolist(), w.tables.tolist(), *part)
    within(out[:, heads].cpu().double(), lse[:, heads].cpu().double(), o, z, spread, amp, dtype, D, 8900, "look-ups")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_widest_masks(dtype):
    """Masks of 64 words, any bits in them, for a tree that is longer than they are; a mask with words to spare."""
    say("tree mask words", dtype)
    w = World([4200, 70], 64, 1, 64, seed=174)
    check_tree(w, [4100, 70], [4200, 70], dtype, 1, words=64, kind="any", seed=6)
    w = World([100, 9], 16, 1, 128, seed=175)
    check_tree(w, [3, 9], [100, 9], dtype, 2, words=64, seed=7)


def test_attend_views_of_a_fused_projection():
    """Queries that are a slice of a wider row, outputs in a wider buffer, tables with a longer row, tokens of both in an
    order of heads first."""
    say("tree views")
    w = World([300, 40], 16, 2, 128, seed=176)
    lens, ctx = [20, 9], [300, 40]
    mask = tree_masks(lens, 1, random.Random(8), "tree").cuda()
    cu, c = i32(running(lens)).cuda(), i32(ctx).cuda()
    wide = w.heads(29, 12, "bf16").cuda()
    q = wide[:, 3:11]
    cache, tab = w.cache(), torch.full((2, w.tables.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    tab[:, :w.tables.shape[1]] = w.tables.cuda()
    want, lse = mr.attend_tree_kv8(q.contiguous(), cu, c, mask, w.tables.cuda(), *cache, return_lse=True)
    room = torch.full((8, 31, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out = room.transpose(0, 1)[1:30]
    got, z = mr.attend_tree_kv8(q, cu, c, mask, tab[:, :w.tables.shape[1]], *cache, out=out, return_lse=True)
    assert got is out and torch.equal(out, want) and torch.equal(z, lse)
    assert bool((room[:, 0] == 5.0).all()) and bool((room[:, 30] == 5.0).all())


# ---------------------------------------------------------------- verification ------------------
def verify(target, ids, parents, cu, ua, un, draft):
    got = mr.verify_tree(target, i32(ids).cuda(), None if parents is None else i32(parents).cuda(), i32(cu).cuda(), ua.cuda(), un.cuda(),
                         draft_probs=draft)
    want = ref.verify_tree(target.float().cpu().numpy(), ids, parents, cu, ua.tolist(), un.tolist(),
                           None if draft is None else draft.float().cpu().numpy())
    assert [x.tolist() for x in got] == list(want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 3, 511, 512, 513, (1 << 20) + 3])
@pytest.mark.parametrize("drawn", [False, True])
def test_verify_vocabularies(dtype, vocab, drawn):
    say("verify vocabulary", dtype, vocab, drawn)
    g = torch.Generator().manual_seed(vocab)
    rng = random.Random(vocab)
    lens = [1, 4, 0, 6]
    T, cu = sum(lens), running(lens)
    make = lambda: torch.softmax(torch.randn(T, vocab, generator=g) * 4, 1).to(TORCH_DT[dtype]).cuda()
    target, draft = make(), make() if drawn else None
    best = target.float().topk(min(vocab, 3), 1).indices.tolist()
    ids = [rng.choice(best[max(t - 1, 0)]) for t in range(T)]
    parents = sum((random_tree(n, rng, 0.5) for n in lens), [])
    for par in (parents, None):
        verify(target, ids, par, cu, torch.rand(T, generator=g), torch.rand(len(lens), generator=g), draft)


def test_verify_rows_past_two_gib():
    """Distributions whose rows begin past 2^31 elements of their buffers."""
    say("verify far rows")
    vocab, stride = 3001, (1 << 30) + 5
    g = torch.Generator().manual_seed(9)
    rows = [torch.softmax(torch.randn(4, vocab, generator=g) * 3, 1).bfloat16().cuda() for _ in range(2)]
    room = torch.empty(2, 3 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    far = [torch.as_strided(r, (4, vocab), (stride, 1)) for r in room]
    for a, b in zip(far, rows):
        a.copy_(b)
    ids = [0] + rows[1][:3].float().argmax(1).tolist()
    u, un = torch.tensor([0.5, 0.1, 0.2, 0.3]).cuda(), torch.tensor([0.6]).cuda()
    for par in (None, i32([-1, 0, 0, 1]).cuda()):
        want = mr.verify_tree(rows[0], i32(ids).cuda(), par, i32([0, 4]).cuda(), u, un, draft_probs=rows[1])
        got = mr.verify_tree(far[0], i32(ids).cuda(), par, i32([0, 4]).cuda(), u, un, draft_probs=far[1])
        assert [x.tolist() for x in got] == [x.tolist() for x in want]
    del room


# ---------------------------------------------------------------- keep --------------------------
def test_keep_head_major_and_far():
    """Heads before rows, in a pool whose pages lie past 2^31 bytes: what a small pool holds afterwards, bit for bit."""
    say("keep far")
    w = World([90, 40], 16, 2, 256, seed=177)
    lens, past = [40, 20], [50, 20]
    kept, path = random_paths(lens, random.Random(2), 3)
    kept[0], path[:40] = 8, [0, 1, 4, 9, 10, 15, 22, 39] + [-1] * 32
    big_n = (1 << 31) // (16 * 2 * 256) + 100
    move = big_n - w.nb
    far = []
    for x in w.cache()[:2]:
        y = torch.zeros(big_n, 2, 16, 256, dtype=torch.uint8, device="cuda").transpose(1, 2)
        y[move:] = x.view(torch.uint8)
        far.append(y)
    scales = [torch.ones(big_n, 2, device="cuda") for _ in range(2)]
    for a, b in zip(scales, (w.ks, w.vs)):
        a[move:] = b.cuda()
    tables = torch.where(w.tables >= 0, w.tables + move, w.tables).cuda()
    mr.keep_kv8(i32(kept).cuda(), i32(path).cuda(), i32(running(lens)).cuda(), i32(past).cuda(), tables, [(*far, *scales)])
    ref.keep(kept, path, running(lens), past, w.tables.tolist(), w.kc, w.ks)
    ref.keep(kept, path, running(lens), past, w.tables.tolist(), w.vc, w.vs)
    assert torch.equal(scales[0][move:].cpu(), w.ks) and torch.equal(scales[1][move:].cpu(), w.vs)
    assert same_codes(far[0][move:].contiguous().view(F8), w.kc) and same_codes(far[1][move:].contiguous().view(F8), w.vc)
    assert all(int(x[:move].count_nonzero()) == 0 for x in far) and all(bool((x[:move] == 1).all()) for x in scales)
