"""GPU parity of the 8-bit paged cache against plain 64-bit implementations (kv8_ref): the append calls
code for code, the attention within tolerances derived from its documented precision."""
import math

import pytest
import torch

import canvas_rope_rotary_amd as mr
import kv8_ref as ref
from gpu_util import TORCH_DT, say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
# what the probabilities (and fp32 queries) are kept to, relative to their size
KEPT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -12, "f32": 2.0 ** -20}


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def bits(t):
    return t.cpu().view(torch.uint8) if t.dtype == F8 else t.cpu()


def same_codes(got, want):
    """e4m3 caches code for code; every NaN code counts as the same."""
    a, b = bits(got), want.view(torch.uint8)
    nan = ((a & 0x7f) == 0x7f) & ((b & 0x7f) == 0x7f)
    return bool(((a == b) | nan).all())


class World:
    """A pool with sequences of `lens` positions in shuffled pages; `extra` pages to spare."""

    def __init__(self, lens, bs=16, hk=2, D=256, seed=0, extra=3, amp=1.0, width=None):
        self.g = torch.Generator().manual_seed(seed)
        need = [-(-n // bs) for n in lens]
        self.nb, self.bs, self.hk, self.D = sum(need) + extra, bs, hk, D
        perm = torch.randperm(self.nb, generator=self.g).int()
        self.tables = torch.full((len(lens), width or max(1, max(need, default=1))), -1, dtype=torch.int32)
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = perm[at:at + k]
            at += k
        codes = (torch.randn(2, self.nb, bs, hk, D, generator=self.g) * 100).clamp(-448, 448).to(F8)
        self.kc, self.vc = codes[0].clone(), codes[1].clone()
        e = torch.randint(-9, -4, (2, self.nb, hk), generator=self.g).float()
        self.ks, self.vs = torch.exp2(e[0]) * amp, torch.exp2(e[1])

    def heads(self, T, h, dtype, scale=1.0):
        return (torch.randn(T, h, self.D, generator=self.g) * scale).to(TORCH_DT[dtype])

    def cache(self):
        return [x.clone().cuda() for x in (self.kc, self.vc, self.ks, self.vs)]


# ---------------------------------------------------------------- append ------------------------
def check_append(w, lens, past, dtype, hq=8, decode=False, amount=None, scale=1.0, q=None, k=None, v=None, pad=0, what=""):
    """One apply_kv8 (or decode_kv8) against the reference; returns the device caches."""
    T = sum(lens)
    q = w.heads(T + pad, hq, dtype) if q is None else q
    k = w.heads(T + pad, w.hk, dtype, scale) if k is None else k
    v = w.heads(T + pad, w.hk, dtype, scale) if v is None else v
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    kc, vc, ks, vs = w.cache()
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    if decode:
        planes = (i32(past) - i32(amount)).expand(3, T)
        mr.decode_kv8(qd, kd, vd, i32(past).cuda(), i32(amount).cuda(), w.tables.cuda(), kc, vc, ks, vs)
    else:
        planes = torch.randint(-1, 5000, (3, T + pad), generator=w.g, dtype=torch.int32)
        mr.apply_kv8(qd, kd, vd, planes.cuda(), i32(cu).cuda(), w.tables.cuda(), kc, vc, ks, vs, pos_offset=i32(past).cuda())
    torch.cuda.synchronize()
    kr, vr = ref.rotate(k[:T], planes[:, :T]), v[:T].float()
    for s, n in enumerate(lens):
        if past[s] >= 0:
            ref.append(kr[cu[s]:cu[s + 1]], w.kc, w.ks, w.tables[s].tolist(), past[s])
            ref.append(vr[cu[s]:cu[s + 1]], w.vc, w.vs, w.tables[s].tolist(), past[s])
    qr = ref.rotate(q[:T], planes[:, :T])
    # the reference's cos and sin and the kernel's differ by some 1e-16, so a rounding may fall one way
    # and the other: one step of the type (fp16: below 2^-14 a step is 2^-24, whatever the value's size)
    off = (qd[:T].cpu().double() - qr.double()).abs() - 2 * HALF_STEP[dtype] * qr.double().abs()
    assert bool((off <= (2.0 ** -24 if dtype == "f16" else 1e-12)).all()), (what, float(off.max()))
    assert torch.equal(qd[T:].cpu(), q[T:]), what
    assert torch.equal(ks.cpu(), w.ks) and torch.equal(vs.cpu(), w.vs), what
    assert same_codes(kc, w.kc) and same_codes(vc, w.vc), what
    return kc, vc, ks, vs


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hk,hq,bs", [(256, 2, 8, 16), (256, 3, 6, 64), (128, 4, 16, 32), (64, 1, 1, 16), (64, 5, 5, 64), (256, 1, 64, 32)])
def test_append_prefill(dtype, D, hk, hq, bs):
    say("append", dtype, D, hk, hq, bs)
    lens = [1, 0, bs, bs + 1, 2 * bs - 1, 0, 70, 5, 0]
    past = [0, 7, 0, bs - 1, 3, 0, 2 * bs + 5, bs - 2, 0]
    w = World([a + b for a, b in zip(lens, past)], bs, hk, D, seed=D + bs)
    check_append(w, lens, past, dtype, hq)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,bs", [(256, 16), (128, 64), (64, 32)])
def test_append_decode(dtype, D, bs):
    say("decode", dtype, D, bs)
    past = [0, 1, bs - 1, bs, 3 * bs + 7, 100, 2 * bs - 1]
    w = World([p + 1 for p in past], bs, 2, D, seed=bs)
    check_append(w, [1] * len(past), past, dtype, decode=True, amount=[0, 58, 0, 56, 58, -3, 0])


@pytest.mark.parametrize("step", [1e-3, 1.0, 40.0])
def test_append_grows_scales(step):
    """Tokens one by one and in pieces, each larger (or smaller) than the last: rows already in a page go
    to the new scale, code for code."""
    w = World([41, 41], 16, 2, 256, seed=3)
    kc = None
    for i, n in enumerate((1, 1, 1, 6, 1, 20, 1, 10)):
        past = [0, 1, 2, 3, 9, 10, 30, 31][i]
        say("grow", step, i)
        kc, vc, ks, vs = check_append(w, [n, n], [past, past], "f32", scale=step ** i if i else 1.0)


def test_append_values():
    """Zeros, values next to the scale's border, subnormal codes, infinities and NaN, the largest and the
    smallest floats."""
    w = World([16] * 6, 16, 1, 64, seed=4)
    k = w.heads(96, 1, "f32")
    v = w.heads(96, 1, "f32")
    v[:16] = 0.0
    v[16:32] = 448.0
    v[32:48] = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9))
    v[48:64, 0, ::3] = math.inf
    v[48:64, 0, 1::7] = math.nan
    v[64:80] *= 2.0 ** -120
    v[80:96] = torch.finfo(torch.float32).max
    k[0:16, 0, 40:] = math.nan
    check_append(w, [16] * 6, [0] * 6, "f32", 1, k=k, v=v)


def test_append_skips_what_has_no_page():
    """Pages outside the pool, positions past the table, negative offsets, padding tokens, empty calls."""
    w = World([40, 40, 40], 16, 2, 128, seed=5)
    w.tables[0, 1] = -1
    w.tables[1, 0] = w.nb
    check_append(w, [40, 40, 30], [0, 0, -5], "bf16", pad=9)
    check_append(w, [10, 3, 20], [40, 45, 45], "bf16", what="past the table")
    kc, vc, ks, vs = w.cache()
    e = lambda h: torch.empty(0, h, 128, dtype=torch.bfloat16, device="cuda")
    mr.apply_kv8(e(8), e(2), e(2), torch.empty(3, 0, dtype=torch.int32, device="cuda"), i32([0, 0, 0, 0]).cuda(), w.tables.cuda(),
                 kc, vc, ks, vs)
    none = torch.empty(0, 16, 2, 128, device="cuda").to(F8)
    q = w.heads(3, 8, "bf16").cuda()
    k = w.heads(3, 2, "bf16").cuda()
    q0 = q.clone()
    mr.decode_kv8(q, k, k, i32([0, 1, 2]).cuda(), i32([0, 0, 0]).cuda(), w.tables.cuda(), none, none, torch.empty(0, 2, device="cuda"),
                  torch.empty(0, 2, device="cuda"))
    planes = i32([0, 1, 2]).expand(3, 3)
    assert torch.allclose(q.cpu().double(), ref.rotate(q0.cpu(), planes).double(), rtol=2.0 ** -7, atol=1e-12)


def test_append_strided():
    """Heads taken out of a fused projection, and a cache with its heads before its rows."""
    T, D = 37, 256
    w = World([T], 16, 2, D, seed=6)
    fused = w.heads(T, 12, "bf16").cuda()
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    kin, vin = k.clone().cpu(), v.clone().cpu()
    planes = torch.randint(0, 99, (3, T), generator=w.g, dtype=torch.int32)
    turned = [x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).cuda() for x in (w.kc.view(torch.uint8), w.vc.view(torch.uint8))]
    turned = [torch.empty_strided(x.shape, (2 * 16 * D, D, 16 * D, 1), dtype=torch.uint8, device="cuda").copy_(x) for x in turned]
    ks, vs = w.ks.cuda(), w.vs.cuda()
    mr.apply_kv8(q, k, v, planes.cuda(), i32([0, T]).cuda(), w.tables.cuda(), *turned, ks, vs)
    ref.append(ref.rotate(kin, planes), w.kc, w.ks, w.tables[0].tolist(), 0)
    ref.append(vin.float(), w.vc, w.vs, w.tables[0].tolist(), 0)
    assert same_codes(turned[0].contiguous().view(F8), w.kc) and same_codes(turned[1].contiguous().view(F8), w.vc)
    assert torch.equal(ks.cpu(), w.ks) and torch.equal(vs.cpu(), w.vs)
    assert torch.equal(k.cpu(), kin) and torch.equal(v.cpu(), vin)


def test_append_many_sequences():
    """The wave search over sequences past one level, with empty ones between."""
    g = torch.Generator().manual_seed(8)
    lens = [int(x) for x in torch.randint(0, 4, (5000,), generator=g)]
    past = [int(x) for x in torch.randint(0, 20, (5000,), generator=g)]
    w = World([a + b for a, b in zip(lens, past)], 16, 1, 64, seed=9)
    check_append(w, lens, past, "bf16", 1)


# ---------------------------------------------------------------- attention ---------------------
def check_attend(w, q_lens, ctx, dtype, hq, *, one=False, softmax_scale=None, q=None, scale=1.0, pad=0, what="", call=None):
    T = sum(q_lens)
    q = w.heads(T + pad, hq, dtype, scale) if q is None else q
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    out = torch.full_like(q, 7.0).cuda()
    lse = torch.full((T + pad, hq), 7.0, device="cuda")
    args = (q.cuda(), None if one else i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache())
    (call or mr.attend_kv8)(*args, softmax_scale=softmax_scale, out=out, lse=lse)
    torch.cuda.synchronize()
    o, z, spread, amp = ref.attend(q[:T], None if one else cu, ctx, w.tables.tolist(), w.kc, w.vc, w.ks, w.vs, softmax_scale)
    got, gz = out[:T].cpu().double(), lse[:T].cpu().double()
    D, n = q.shape[2], max(list(ctx) + [1])
    # scores: up to three exact terms a product, summed in fp32 (3 D roundings at most), then the factor;
    # fp32 queries are kept to KEPT.  exp2 and the sums of p add some 2^-21 and n 2^-24.
    ds = ((3 * D + 8) * 2.0 ** -24 + (KEPT["f32"] if dtype == "f32" else 0)) * amp
    tol = HALF_STEP[dtype] * o.abs() * 1.01 + (2 * ds[..., None] + KEPT[dtype] + 2.0 ** -20 + 2 * n * 2.0 ** -24) * spread + 1e-30
    bad = ~((got - o).abs() <= tol) & ~(torch.isnan(got) & torch.isnan(o))
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got - o).abs() / tol)[bad].max()), bad.nonzero()[:4].tolist())
    fin = torch.isfinite(z)
    assert torch.equal(fin, torch.isfinite(gz)) and torch.equal(torch.isnan(z), torch.isnan(gz)), what
    dz = (gz[fin] - z[fin]).abs()
    assert bool((dz <= ds[fin] + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * z[fin].abs()).all()), (what, float(dz.max()))
    empty = torch.isneginf(z)
    assert bool((got[empty] == 0).all()), what
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all()), what
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hq,hk,bs", [(256, 8, 2, 16), (256, 6, 3, 64), (128, 16, 4, 32), (64, 4, 4, 16), (64, 64, 1, 64), (256, 16, 1, 32)])
def test_attend_one_token(dtype, D, hq, hk, bs):
    say("attend 1", dtype, D, hq, hk, bs)
    ctx = [1, 2, 15, 16, 17, 31, 33, 110, 129, 300, 0, 64, 511, 513]
    w = World(ctx, bs, hk, D, seed=D + hq)
    check_attend(w, [1] * len(ctx), ctx, dtype, hq, one=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hq,hk,bs", [(256, 8, 2, 16), (128, 16, 4, 64), (64, 3, 3, 32), (256, 4, 4, 16), (128, 14, 2, 16)])
def test_attend_ragged(dtype, D, hq, hk, bs):
    """Prompts, pieces of prompts and single tokens in one call; rows that see nothing."""
    say("attend ragged", dtype, D, hq, hk, bs)
    q_lens = [1, 0, 2, 5, 33, 70, 1, 16, 3, 0, 4]
    ctx = [200, 5, 2, 40, 33, 131, 0, 90, 1, 0, 67]  # the sixth-last has no context, the third-last less than its tokens
    w = World(ctx, bs, hk, D, seed=D + hq + 1)
    check_attend(w, q_lens, ctx, dtype, hq, pad=5)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,hq,hk", [(256, 8, 2), (128, 8, 1), (64, 2, 2)])
def test_attend_prompts(dtype, D, hq, hk):
    """Longer prompts: several tiles of rows, tiles that end inside a page, a piece on a long cache."""
    say("attend prompts", dtype, D, hq, hk)
    q_lens, ctx = [150, 67, 129], [150, 300, 129 + 16]
    w = World(ctx, 16, hk, D, seed=D + hq + 2)
    check_attend(w, q_lens, ctx, dtype, hq)


@pytest.mark.parametrize("dtype,hq,hk,D", [("bf16", 8, 2, 256), ("f32", 4, 2, 128), ("f16", 2, 1, 64)])
@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_attend_long(dtype, hq, hk, D, q_len):
    """A long axis split over workgroups and joined, next to a short sequence in a wide table."""
    say("attend long", dtype, q_len)
    ctx = [9001, 50, 4096]
    w = World(ctx, 64, hk, D, seed=11)
    check_attend(w, [q_len] * 3, ctx, dtype, hq, one=q_len == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_seqs,hq,hk,D", [(70, 8, 2, 64), (300, 6, 3, 128), (4300, 2, 1, 64)])
def test_attend_uneven_batch(dtype, n_seqs, hq, hk, D):
    """More sequences than lanes (and than lanes squared), contexts from none to thousands: the long ones
    are cut, the short ones are not, and both kinds lie side by side in the batch."""
    say("attend uneven", dtype, n_seqs, D)
    g = torch.Generator().manual_seed(n_seqs)
    ctx = torch.randint(0, 60, (n_seqs,), generator=g)
    ctx[torch.randint(0, n_seqs, (9,), generator=g)] = torch.randint(1500, 6000, (9,), generator=g)
    ctx[0], ctx[-1], ctx[n_seqs // 2] = 3001, 2500, 0
    ctx = ctx.tolist()
    w = World(ctx, 16, hk, D, seed=n_seqs)
    check_attend(w, [1] * n_seqs, ctx, dtype, hq, one=True)
    q_lens = [1 + (s % 3) if c else s % 2 for s, c in enumerate(ctx)]
    check_attend(w, q_lens, ctx, dtype, hq, pad=3)


@pytest.mark.parametrize("dtype,D,n_seqs", [("bf16", 256, 64), ("f16", 64, 65), ("bf16", 128, 130), ("f32", 64, 7)])
def test_attend_many_prompts(dtype, D, n_seqs):
    """Prompts by the length of their contexts (up to as many sequences as lanes) and in the batch's order
    (more), some of one token or none, some on a cache, some with fewer positions than tokens."""
    say("attend many prompts", dtype, D, n_seqs)
    g = torch.Generator().manual_seed(n_seqs)
    q_lens = torch.randint(5, 45, (n_seqs,), generator=g).tolist()
    q_lens[1], q_lens[2], q_lens[n_seqs // 2], q_lens[-1] = 0, 1, 130, 77
    past = [int(x) for x in torch.randint(0, 90, (n_seqs,), generator=g)]
    past[3], past[4] = -3, 700
    ctx = [max(a + b, 0) for a, b in zip(q_lens, past)]
    w = World(ctx, 32, 2, D, seed=n_seqs + D)
    check_attend(w, q_lens, ctx, dtype, 12, pad=9)


@pytest.mark.parametrize("one", [True, False])
def test_attend_long_chunks(one):
    """So many KV heads and long sequences that a workgroup's chunk passes 4,096 tokens (its pages are
    looked up again), on tables that name the same pages over and over."""
    say("attend long chunks", one)
    w = World([640], 16, 64, 64, seed=19)
    ctx = [8900] * 7 + [70, 8889]
    w.tables = w.tables[:, :40].repeat(9, 15)
    w.tables[1] = w.tables[1].flip(0)
    cu = list(range(10)) if one else [0, 2, 3, 4, 5, 6, 7, 8, 8, 11]
    q = w.heads(cu[-1], 64, "bf16")
    out, lse = mr.attend_kv8(q.cuda(), None if one else i32(cu).cuda(), i32(ctx).cuda(), w.tables.cuda(), *w.cache(), return_lse=True)
    heads = [0, 31, 63]
    part = [x[:, :, heads] for x in (w.kc, w.vc)] + [x[:, heads] for x in (w.ks, w.vs)]
    o, z, spread, amp = ref.attend(q[:, heads], None if one else cu, ctx, w.tables.tolist(), *part, None)
    ds = (3 * 64 + 8) * 2.0 ** -24 * amp
    tol = HALF_STEP["bf16"] * o.abs() * 1.01 + (2 * ds[..., None] + KEPT["bf16"] + 2.0 ** -20 + 2 * 8900 * 2.0 ** -24) * spread + 1e-30
    assert bool(((out[:, heads].cpu().double() - o).abs() <= tol).all())
    assert bool(((lse[:, heads].cpu().double() - z).abs() <= ds + 8900 * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * z.abs()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 6, 70])
def test_attend_ignores_what_is_not_seen(dtype, q_len):
    """NaN codes, NaN and infinite scales, and bad page numbers wherever a row does not look; NaN in later
    tokens' keys and values reaches no earlier row, and does reach the rows that see them."""
    say("attend unseen", dtype, q_len)
    ctx = [100, 37, 0, 70]
    w = World([128, 64, 16, 80], 16, 2, 256, seed=12, width=9)
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
    check_attend(w, [q_len, min(q_len, 37), 1, q_len], ctx, dtype, 8, one=q_len == 1, what="behind the end")
    # position 95 and 60 hold NaN in one head's value and another's key
    p = int(w.tables[0, 95 // 16])
    w.vc.view(torch.uint8)[p, 95 % 16, 0, 5] = 0x7f
    w.vc.view(torch.uint8)[p, 95 % 16, 0, 201] = 0xff
    p = int(w.tables[3, 60 // 16])
    w.kc.view(torch.uint8)[p, 60 % 16, 1, 9] = 0x7f
    check_attend(w, [q_len, min(q_len, 37), 1, q_len], ctx, dtype, 8, one=q_len == 1, what="NaN in a later token")


def test_attend_holes():
    """A page of the middle that is missing is not attended to; a row with missing pages only is empty."""
    w = World([100, 40, 33], 16, 2, 128, seed=13)
    w.tables[0, 2] = -1
    w.tables[0, 6] = -1
    w.tables[1, :] = -1
    w.tables[2, 1] = w.nb + 5
    for q_len in (1, 2, 33):
        check_attend(w, [q_len] * 3, [100, 40, 33], "bf16", 8, one=q_len == 1, what=q_len)


def test_attend_scores():
    """Large scores (one key takes everything), equal scores, a negative and a zero factor, zero and
    infinite queries."""
    w = World([200, 90], 16, 2, 256, seed=14)
    check_attend(w, [1, 1], [200, 90], "bf16", 8, one=True, scale=60.0)
    check_attend(w, [50, 20], [200, 90], "bf16", 8, scale=60.0)
    for f in (0.0, -0.05, 1.0):
        check_attend(w, [3, 1], [200, 90], "f32", 8, softmax_scale=f)
        check_attend(w, [40, 33], [200, 90], "f32", 8, softmax_scale=f)
    q = w.heads(73, 8, "bf16")
    q[::2] = 0
    check_attend(w, [40, 33], [200, 90], "bf16", 8, q=q)
    q = w.heads(73, 8, "f32")
    q[5, 3] *= 1e-30
    q[6, 2] *= 1e-42
    q[50, 1] = 0
    check_attend(w, [40, 33], [200, 90], "f32", 8, q=q)
    q[:, 0, 10] = math.inf
    q[:, 1, 3] = math.nan
    out, _ = mr.attend_kv8(q.cuda(), i32([0, 40, 73]).cuda(), i32([200, 90]).cuda(), w.tables.cuda(), *w.cache())
    assert bool(torch.isnan(out[:, :2]).all()) and bool(torch.isfinite(out[:, 2:]).all())


def test_attend_strided_and_workspace():
    """Q and out as views, the caller's workspace, refused workspaces."""
    w = World([700, 20], 16, 2, 128, seed=15)
    big = w.heads(2, 24, "bf16").cuda()
    q, out = big[:, 3:11], torch.zeros(2, 16, 128, dtype=torch.bfloat16, device="cuda")[:, 4:12]
    tab, cache = w.tables.cuda(), w.cache()
    n = mr.attend_kv8_workspace_bytes(q, 2, tab, cache[0], True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mr.attend_kv8(q, None, i32([700, 20]).cuda(), tab, *cache, out=out, workspace=ws)
    o, _, spread, _ = ref.attend(q.cpu(), None, [700, 20], w.tables.tolist(), w.kc, w.vc, w.ks, w.vs)
    assert bool(((out.cpu().double() - o).abs() <= 2.0 ** -7 * spread + 1e-9).all())
    with pytest.raises(mr.MropeError):
        mr.attend_kv8(q, None, i32([700, 20]).cuda(), tab, *cache, workspace=ws[:n - 256])
    with pytest.raises(ValueError):
        mr.attend_kv8(q, None, i32([700, 20]).cuda(), tab, *cache, workspace=ws.view(torch.int32))


def test_binding_refusals():
    w = World([20, 20], 16, 2, 128, seed=16)
    kc, vc, ks, vs = w.cache()
    tab, q, k = w.tables.cuda(), w.heads(2, 8, "bf16").cuda(), w.heads(2, 2, "bf16").cuda()
    one = i32([1, 1]).cuda()
    bad = [
        dict(block_tables=tab.long()), dict(block_tables=tab[:1]), dict(k_cache=kc.float()), dict(k_cache=kc[:, :, :1]),
        dict(v_cache=vc[1:]), dict(k_scale=ks.half()), dict(v_scale=vs[:, :1]), dict(context_lens=one.long()),
        dict(context_lens=one[:1]), dict(q=q.cpu()), dict(out=q[:1]), dict(lse=torch.empty(2, 7, device="cuda")),
    ]
    base = dict(q=q, cu_seqlens=None, context_lens=one, block_tables=tab, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            mr.attend_kv8(**{**base, **kw})
    with pytest.raises(TypeError):
        mr.attend_kv8(**{**base, "q": q.double()})
    with pytest.raises(mr.MropeError):
        mr.attend_kv8(**{**base, "q": q[:, :7]})
    dec = dict(q=q, k=k, v=k, pos=one, amount=one, block_tables=tab, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)
    for kw in (dict(v=k[:, :1]), dict(v=k.float()), dict(pos=one.long()), dict(k_cache=kc.to(torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            mr.decode_kv8(**{**dec, **kw})
    app = dict(q=q, k=k, v=k, planes_=torch.zeros(3, 2, dtype=torch.int32, device="cuda"), cu_seqlens=i32([0, 1, 2]).cuda(), block_tables=tab,
               k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)
    for kw in (dict(planes_=torch.zeros(3, 1, dtype=torch.int32, device="cuda")), dict(cu_seqlens=i32([0, 2]).cuda()), dict(pos_offset=one[:1])):
        with pytest.raises((ValueError, TypeError)):
            mr.apply_kv8(**{**app, **kw})


def test_graph_replay_and_streams():
    """A decode step captured and replayed with new inputs, eager work between the replays; two graphs of
    the same call; the same calls on a side stream; a prepared call."""
    w = World([400, 77], 16, 2, 256, seed=17)
    cache = w.cache()
    tab = w.tables.cuda()
    q, k, v = (w.heads(2, h, "bf16").cuda() for h in (8, 2, 2))
    pos, amount, ctx = i32([390, 60]).cuda(), i32([58, 0]).cuda(), i32([391, 61]).cuda()
    out = torch.empty_like(q)

    def step():
        mr.decode_kv8(q, k, v, pos, amount, tab, *cache)
        mr.attend_kv8(q, None, ctx, tab, *cache, out=out)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    side = torch.cuda.Stream()
    for i in range(6):
        new = [w.heads(2, h, "bf16").cuda() for h in (8, 2, 2)]
        state = [x.clone() for x in cache]

        def put():
            for a, b in zip((q, k, v), new):
                a.copy_(b)
            for a, b in zip(cache, state):
                a.view(torch.uint8).copy_(b.view(torch.uint8))

        put()
        step()
        want, codes = out.clone(), [bits(x).clone() for x in cache]
        torch.cuda.synchronize()
        put()
        out.zero_()
        if i < 4:
            graphs[i % 2].replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want), i
        assert all(torch.equal(bits(a), b) for a, b in zip(cache, codes)), i
        torch.ones(1 << 20, device="cuda").sum().item()  # eager work between the replays
    run = mr.prepare(mr.attend_kv8, q, None, ctx, tab, *cache, out=out)
    for _ in range(3):
        q.copy_(w.heads(2, 8, "bf16"))
        want = mr.attend_kv8(q, None, ctx, tab, *cache)[0]
        out.zero_()
        junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        run()
        assert torch.equal(out, want)
        del junk
