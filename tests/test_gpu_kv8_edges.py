"""The 8-bit cache's calls at the edges of what their documentation allows."""
import math

import pytest
import torch

import canvas_rope_rotary_amd as mr
import kv8_ref as ref
from gpu_util import say
from test_gpu_kv8 import F8, HALF_STEP, World, check_append, i32, same_codes

pytestmark = pytest.mark.gpu
KEPT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -16, "f32": 2.0 ** -24}
I32 = 2 ** 31 - 1


def check(w, cu, ctx, q, dtype, n, *, softmax_scale=None, out=None, cache=None, extra=0.0, what=""):
    """attend_kv8 on World w against 64 bits: tolerances of the documented precision (a score: at most three
    exact terms a product, each sum rounded; l and the output: n positions of at most three terms; exp2 an
    ulp; `extra` of the spread where a test's numbers need it).  Rows behind cu's last are left alone."""
    T, D = (q.shape[0] if cu is None else cu[-1]), q.shape[2]
    o_dev = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    mr.attend_kv8(q.cuda(), None if cu is None else i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *(cache or w.cache()),
                  softmax_scale=softmax_scale, out=o_dev, lse=lse)
    o, z, spread, amp = ref.attend(q[:T], cu, ctx, w.tables.tolist(), w.kc, w.vc, w.ks, w.vs, softmax_scale)
    got, gz = o_dev[:T].cpu().double(), lse[:T].cpu().double()
    ds = ((3 * D + 8) * 2.0 ** -24 + (2.0 ** -24 if dtype == "f32" else 0)) * amp
    tol = HALF_STEP[dtype] * o.abs() * 1.01 + (2 * ds[..., None] + KEPT[dtype] + 2.0 ** -22 + (4 * n + 4) * 2.0 ** -24 + extra) * spread
    tol += 2.0 ** -24 if dtype == "f16" else 2.0 ** -120
    bad = ~((got - o).abs() <= tol) & ~(torch.isnan(got) & torch.isnan(o))
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), o[bad][:4].tolist())
    fin = torch.isfinite(z)
    assert torch.equal(fin, torch.isfinite(gz)), what
    dz = (gz[fin] - z[fin]).abs()
    assert bool((dz <= ds[fin] + (n + 4) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * z[fin].abs()).all()), (what, float(dz.max()))
    assert bool((got[~fin] == 0).all()), what
    assert bool((o_dev[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all()), what


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n_seqs", [5, 70])
def test_lengths_past_the_table(dtype, n_seqs):
    """Lengths at the top of int32 (every position of the table is seen), next to none and negative ones,
    for prompts (ranked by length up to 64 sequences) and for single tokens."""
    say("past the table", dtype, n_seqs)
    w = World([96] * n_seqs, 16, 2, 64, seed=n_seqs)
    lens = ([40, 150, 0, 1, 77] * 14)[:n_seqs]
    ctx = ([I32, 0, 5, I32 - 1, 90] * 14)[:n_seqs]
    ctx[-1] = -I32 - 1
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    check(w, cu, ctx, w.heads(cu[-1] + 3, 6, dtype), dtype, 96, what="prompts")
    check(w, None, ctx, w.heads(n_seqs, 6, dtype), dtype, 96, what="tokens")
    check(w, list(range(n_seqs + 1)), ctx, w.heads(n_seqs + 2, 6, dtype), dtype, 96, what="tokens by cu")


def prompts_and_tokens(w, n, hq, dtype, what, q=None, lens=(90, 60), softmax_scale=None, extra=0.0):
    """The World's first two sequences of n positions as pieces of prompts and as single tokens."""
    cu = [0, lens[0], sum(lens)]
    q = w.heads(cu[-1], hq, dtype) if q is None else q
    check(w, cu, [n] * 2, q, dtype, n, softmax_scale=softmax_scale, extra=extra, what=(what, "prompts"))
    check(w, None, [n] * 2, q[[7, cu[-1] - 1]], dtype, n, softmax_scale=softmax_scale, extra=extra, what=(what, "tokens"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [256, 64])
def test_value_scales_side_by_side(dtype, D):
    """Pages of V whose scales differ by up to 2^216: zero pages (as an append leaves them) next to large ones,
    and both ends of the range; scores that rise along the context, so that the running maximum follows."""
    say("value scales", dtype, D)
    for case, exps in enumerate(((-96, 0, 30), (-96, 60), (-96, -96, 118), (-96, -90), (-9, -5, 25), (118, 110, 80))):
        w = World([200, 200], 16, 2, D, seed=case)
        pick = torch.randint(0, len(exps), w.vs.shape, generator=w.g)
        w.vs = torch.exp2(torch.tensor(exps)[pick].float())
        zero = (w.vs == 2.0 ** -96) & (len(set(exps)) > 1)
        w.vc.view(torch.uint8)[zero[:, None, :, None].expand_as(w.vc)] = 0
        w.vc = w.vc.float().clamp(-255, 255).to(F8)  # (at 2^118 to 2^126)
        prompts_and_tokens(w, 200, 4, dtype, exps)
        q = w.heads(150, 4, dtype, 3.0)
        prompts_and_tokens(w, 200, 4, dtype, (exps, "wide scores"), q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_values(dtype):
    """Codes of 448 at a scale of 2^120 (past fp32's largest): rows that do not see them are untouched, and a
    row's average of them is right where it can be held."""
    say("largest values", dtype)
    w = World([100, 100], 16, 2, 128, seed=31)
    for s in range(2):
        page = int(w.tables[s, 5])
        w.vs[page, 1] = 2.0 ** 120
        w.vc.view(torch.uint8)[page, :, 1] = 0x7e
    q = w.heads(150, 4, dtype)
    for cu, qq in (([0, 90, 150], q), (None, q[:2])):
        ctx = [100, 84 + 4]
        out, _ = mr.attend_kv8(qq.cuda(), None if cu is None else i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache())
        o, z, spread, amp = ref.attend(qq, cu, ctx, w.tables.tolist(), w.kc, w.vc, w.ks, w.vs)
        held = o.abs() < 2.0 ** 127
        assert bool(held.any()) and bool((o.abs() > 2.0 ** 100).any())
        ds = (3 * 128 + 9) * 2.0 ** -24 * amp[..., None]
        tol = HALF_STEP[dtype] * o.abs() * 1.01 + (2 * ds + KEPT[dtype] + 2.0 ** -22 + 404 * 2.0 ** -24) * spread
        got = out.cpu().double()
        assert bool(((got - o).abs() <= tol)[held].all()), (cu, float(((got - o).abs() / tol)[held].max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_key_scales(dtype):
    """Pages of K at both ends of the scales' range, under queries that bring the scores back."""
    say("key scales", dtype)
    for case, e in enumerate((-90, -40, 60, 100)):
        w = World([200, 200], 16, 2, 128, seed=40 + case)
        w.ks = w.ks * 2.0 ** e
        w.ks[::3] = 2.0 ** max(e - 30, -96)
        prompts_and_tokens(w, 200, 4, dtype, e, w.heads(150, 4, dtype) * 2.0 ** -e)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("softmax_scale", [1e-18, -1e-20, 1e-30, 1e-44])
def test_tiny_factors(dtype, softmax_scale):
    """Factors so small that with a small page scale they vanish: every position that a row sees weighs the
    same, and those that it does not see weigh nothing."""
    say("tiny factor", dtype, softmax_scale)
    w = World([200, 200], 16, 2, 128, seed=50)
    w.ks.fill_(2.0 ** -96)
    w.kc.view(torch.uint8)[:] = 0
    prompts_and_tokens(w, 200, 4, dtype, "zero keys", softmax_scale=softmax_scale)
    w.ks[1::2] = 2.0 ** -20
    w.kc = (torch.randn(w.kc.shape, generator=w.g) * 100).to(F8)
    prompts_and_tokens(w, 200, 4, dtype, "small keys", softmax_scale=softmax_scale)


def test_output_and_queries_of_one_buffer():
    """Views of one buffer that share no row are taken, those that do are refused and nothing is written."""
    say("one buffer")
    w = World([150, 40], 16, 2, 64, seed=60)
    cu, ctx = [0, 70, 90], [150, 40]
    for what, q_at, o_at in (("heads of a token", (slice(None, 90), slice(0, 4)), (slice(None, 90), slice(4, 8))),
                             ("tokens", (slice(0, 90), slice(0, 4)), (slice(90, 180), slice(2, 6))),
                             ("turns", (slice(0, 180, 2), slice(0, 4)), (slice(1, 180, 2), slice(1, 5))),
                             ("strides", (slice(0, 180, 2), slice(0, 4)), (slice(0, 90), slice(4, 8)))):
        big = w.heads(180, 8, "bf16").cuda()
        q, out = big[q_at], big[o_at]
        out.fill_(7.0)
        check(w, cu, ctx, q.clone().cpu(), "bf16", 150)
        want = mr.attend_kv8(q.clone(), i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache())[0]
        kept = big.clone()
        mr.attend_kv8(q, i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache(), out=out)
        assert torch.equal(out, want), what
        kept[o_at] = want
        assert torch.equal(big, kept), what
    for q_at, o_at in (((slice(0, 90), slice(0, 4)), (slice(0, 90), slice(3, 7))), ((slice(0, 90), slice(0, 4)), (slice(1, 91), slice(0, 4))),
                       ((slice(0, 180, 2), slice(0, 4)), (slice(0, 90), slice(3, 7)))):
        big = w.heads(180, 8, "bf16").cuda()
        kept = big.clone()
        with pytest.raises(mr.MropeError, match="overlap"):
            mr.attend_kv8(big[q_at], i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache(), out=big[o_at])
        assert torch.equal(big, kept)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_head_major_cache(dtype):
    """A cache with its heads before its rows and a gap between pages."""
    say("head-major", dtype)
    w = World([200, 90], 32, 3, 128, seed=70)
    turned = []
    for x in w.cache()[:2]:
        room = torch.zeros(w.nb, 3, 40, 128, dtype=torch.uint8, device="cuda")
        y = room[:, :, :32].transpose(1, 2)
        y.copy_(x.view(torch.uint8))
        turned.append(y)
    cache = (*turned, w.ks.cuda(), w.vs.cuda())
    check(w, [0, 100, 130], [200, 90], w.heads(130, 6, dtype), dtype, 200, cache=cache)
    check(w, None, [200, 90], w.heads(2, 6, dtype), dtype, 200, cache=cache)


@pytest.mark.parametrize("q_len", [1, 60])
def test_pool_past_two_gib(q_len):
    """Pages past 2^31 bytes of a pool hold and give what the same pages of a small pool do, bit for bit."""
    say("large pool", q_len)
    w = World([150, 33], 64, 2, 256, seed=71)
    big_n = 70000  # of 32 KB
    move = big_n - w.nb
    small = w.cache()
    big = [torch.zeros(big_n, *x.shape[1:], dtype=torch.uint8 if x.dtype == F8 else x.dtype, device="cuda") for x in small]
    for a, b in zip(big, small):
        a[move:] = b.view(a.dtype)
    far = torch.where(w.tables >= 0, w.tables + move, w.tables).cuda()
    past = [150 - q_len, 33 - min(q_len, 33)]
    cu = [0, 150 - past[0], 150 - past[0] + 33 - past[1]]
    q, k, v = (w.heads(cu[-1], h, "bf16").cuda() for h in (8, 2, 2))
    planes = torch.randint(0, 200, (3, cu[-1]), generator=w.g, dtype=torch.int32).cuda()
    outs = []
    for cache, tab in ((small, w.tables.cuda()), (big, far)):
        qq = q.clone()
        if q_len == 1:
            mr.decode_kv8(qq, k, v, i32(past).cuda(), i32([0, 3]).cuda(), tab, *cache)
        else:
            mr.apply_kv8(qq, k, v, planes, i32(cu).cuda(), tab, *cache, pos_offset=i32(past).cuda())
        outs.append(mr.attend_kv8(qq, None if q_len == 1 else i32(cu).cuda(), i32([150, 33]).cuda(), tab, *cache, return_lse=True))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for a, b in zip(big, small):
        assert torch.equal(a[move:], b.view(a.dtype)) and int(a[:move].count_nonzero()) == 0


@pytest.mark.parametrize("dtype,D", [("bf16", 256), ("f16", 64), ("f32", 128)])
@pytest.mark.parametrize("n_seqs", [1, 3, 66])
def test_prompts_with_nan_values(dtype, D, n_seqs):
    """NaN codes in V all over a context of many tiles, in whole pieces and cut into chunks: each reaches the rows
    that see it, in its dim, and no other; pages that are missing between them; waves of a tile that see fewer
    tiles than the others."""
    say("nan values", dtype, D, n_seqs)
    n = 37 if n_seqs > 3 else 150
    ctx = [n + (61 * s) % 400 for s in range(n_seqs)]
    w = World(ctx, 16, 2, D, seed=80 + n_seqs)
    for s in range(n_seqs):
        if ctx[s] > 100:
            w.tables[s, 3] = -1
    raw = w.vc.view(torch.uint8)
    hit = torch.rand(raw.shape, generator=w.g) < 3e-5 * 256 / D
    raw[hit] = torch.tensor([0x7f, 0xff], dtype=torch.uint8)[torch.randint(0, 2, (int(hit.sum()),), generator=w.g)]
    cu = [n * s for s in range(n_seqs + 1)]
    check(w, cu, ctx, w.heads(cu[-1], 6, dtype), dtype, max(ctx), what=n_seqs)


def test_prompts_captured_and_on_two_streams():
    """Pieces of prompts (cut and joined, and whole) in a graph, replayed with other inputs and eager work between
    the replays; two such calls at once on streams of their own."""
    say("prompts captured")
    w = World([2100, 900], 16, 2, 128, seed=90)
    tab, cache = w.tables.cuda(), w.cache()
    cu, ctx = i32([0, 40, 130]).cuda(), i32([2100, 900]).cuda()
    q = w.heads(130, 8, "bf16").cuda()
    out, lse = torch.empty_like(q), torch.empty(130, 8, device="cuda")

    def call():
        mr.attend_kv8(q, cu, ctx, tab, *cache, out=out, lse=lse)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        q.copy_(w.heads(130, 8, "bf16"))
        call()
        want = out.clone(), lse.clone()
        out.zero_(), lse.zero_()
        torch.ones(1 << 20, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [w.heads(130, 8, "bf16").cuda() for _ in range(2)]
    want = [mr.attend_kv8(x, cu, ctx, tab, *cache)[0].clone() for x in inputs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(mr.attend_kv8(inputs[k], cu, ctx, tab, *cache)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[k]) for k in range(2) for x in got[k])
