"""GPU tests of the page calls against a model in Python lists, and of a serving loop that uses them with
the append and the attention."""
import random

import pytest
import torch

import canvas_rope_rotary_amd as mr
import kv8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Dev:
    """The same state on the device and in the model, with pools of several shapes and types."""

    def __init__(self, n_pages, n_rows, width, bs, seed=0, odd=False):
        g = torch.Generator().manual_seed(seed)
        self.m = ref.Pages(n_pages, n_rows, width, bs)
        self.refcount = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.tables = torch.full((n_rows, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n_rows, dtype=torch.int32, device="cuda")
        shapes = [((n_pages, bs, 2, 16), torch.uint8), ((n_pages, 2), torch.float32), ((n_pages, bs, 2, 64), torch.bfloat16)]
        if odd:
            shapes += [((n_pages, 7), torch.uint8), ((n_pages,), torch.int32)]
        self.host = [torch.randint(0, 250, s, generator=g).to(t) for s, t in shapes]
        self.pools = [x.cuda() for x in self.host]
        if odd:  # pages with a gap behind them
            gap = torch.zeros(n_pages, 3, bs, dtype=torch.float32)
            gap[:, 1] = torch.randn(n_pages, bs, generator=g)
            self.host.append(gap[:, 1].clone())
            self.pools.append(gap.cuda()[:, 1])

    @property
    def state(self):
        return self.refcount, self.tables, self.lens

    def check(self, what=""):
        assert self.refcount.tolist() == self.m.ref, what
        assert self.tables.tolist() == self.m.tab, what
        assert self.lens.tolist() == self.m.len, what
        for a, b in zip(self.pools, self.host):
            assert torch.equal(a.cpu(), b), what


def test_pages_random_runs():
    """Random sequences of calls, with shortages, repeated and bad rows, forks of forks."""
    for seed in range(6):
        r = random.Random(seed)
        bs = r.choice([1, 16, 64])
        n_rows, n_pages, width = r.choice([(1, 1, 1), (9, 23, 7), (40, 300, 12)])
        d = Dev(n_pages, n_rows, width, bs, seed, odd=seed % 2 == 1)
        for step in range(40):
            op = r.choice(["grow", "grow", "grow", "free", "fork", "fork", "compact"])
            n = r.randrange(0, n_rows + 1)
            rows = [r.randrange(-1, n_rows + 1) if r.random() < 0.1 else r.randrange(n_rows) for _ in range(n)]
            what = (seed, step, op, n)
            if op == "grow":
                lens = [r.choice([-1, 0, r.randrange(0, bs * width + 2), r.randrange(0, bs * 3)]) for _ in rows]
                got = mr.pages_grow(*d.state, i32(rows), i32(lens), bs)
                assert got.tolist() == d.m.grow(rows, lens), what
            elif op == "free":
                rows = rows[:r.randrange(0, 4)]
                mr.pages_free(*d.state, i32(rows))
                d.m.free(rows)
            elif op == "fork":
                dst = [r.randrange(-1, n_rows + 1) if r.random() < 0.1 else r.randrange(n_rows) for _ in rows]
                got = mr.pages_fork(*d.state, i32(rows), i32(dst), bs, d.pools)
                assert got.tolist() == d.m.fork(rows, dst, d.host), what
            else:
                assert mr.pages_compact(*d.state, d.pools).item() == d.m.compact(d.host), what
            d.check(what)


def test_pages_large_pool():
    """More pages than the plan's workgroup ranks at a time, more requests than it has threads."""
    r = random.Random(3)
    d = Dev(50001, 3000, 40, 16, 1)
    rows = list(range(3000))
    r.shuffle(rows)
    lens = [r.randrange(0, 300) for _ in rows]
    assert mr.pages_grow(*d.state, i32(rows), i32(lens), 16).tolist() == d.m.grow(rows, lens)
    d.check("grow")
    gone = rows[500:2400]
    mr.pages_free(*d.state, i32(gone + gone[:7]))
    d.m.free(gone)
    d.check("free")
    src, dst = [rows[i % 500] for i in range(1500)], gone[:1500]
    assert mr.pages_fork(*d.state, i32(src), i32(dst), 16, d.pools).tolist() == d.m.fork(src, dst, d.host)
    d.check("fork")
    mr.pages_free(*d.state, i32(rows[:300]))
    d.m.free(rows[:300])
    assert mr.pages_compact(*d.state, d.pools).item() == d.m.compact(d.host) > 0
    d.check("compact")
    assert mr.pages_compact(*d.state, d.pools).item() == d.m.compact(d.host) == 0


@pytest.mark.parametrize("n_pages,offset", [(20011, 1), (16384, 0), (16401, 3)])
def test_pages_unaligned_counts_and_large_pages(n_pages, offset):
    """Counts that begin off a 16-byte boundary, pools of odd sizes, pages of several spans next to pages of
    a few bytes, a pool that needs the byte path."""
    say("pages unaligned", n_pages, offset)
    r = random.Random(n_pages)
    d = Dev(n_pages, 50, 600, 16, 5)
    store = torch.zeros(n_pages + 8, dtype=torch.int32, device="cuda")
    d.refcount = store[offset:offset + n_pages]
    d.host = [torch.randint(0, 250, (n_pages, n), dtype=torch.uint8) for n in (8, 5001, 1)]
    d.pools = [x.cuda() for x in d.host]
    for step in range(4):
        rows = list(range(50))
        lens = [r.randrange(0, 9000) for _ in rows]
        assert mr.pages_grow(*d.state, i32(rows), i32(lens), 16).tolist() == d.m.grow(rows, lens), step
        gone = r.sample(rows, 30)
        mr.pages_free(*d.state, i32(gone))
        d.m.free(gone)
        src = [x for x in rows if x not in gone][:6]
        got = mr.pages_fork(*d.state, i32(src), i32(gone[:6]), 16, d.pools)
        assert got.tolist() == d.m.fork(src, gone[:6], d.host), step
        mr.pages_free(*d.state, i32(src))
        d.m.free(src)
        assert int(mr.pages_compact(*d.state, d.pools)) == d.m.compact(d.host), step
        d.check(step)
    assert int(store[:offset].abs().sum()) == 0 and int(store[offset + n_pages:].abs().sum()) == 0


def test_pages_shortage_in_order():
    d = Dev(10, 5, 10, 4, 2)
    rows, lens = [0, 1, 2, 3, 4], [8, 20, 16, 0, 4]  # 2, 5, 4 (too many), 0, 1 (behind it)
    assert mr.pages_grow(*d.state, i32(rows), i32(lens), 4).tolist() == [0, 0, 1, 0, 1] == d.m.grow(rows, lens)
    d.check()


def test_pages_copy():
    d = Dev(30, 1, 1, 16, 4, odd=True)
    src, dst = [3, 3, 7, -1, 5, 30, 2], [10, 11, 12, 13, -2, 14, 2]
    mr.pages_copy(i32(src), i32(dst), d.pools)
    for x in d.host:
        x[10], x[11], x[12] = x[3], x[3], x[7]
    d.check()
    mr.pages_copy(i32([]), i32([]), d.pools)


def test_pages_refusals():
    d = Dev(8, 4, 4, 16, 5)
    one = i32([0])
    for bad in (dict(rows=one.long()), dict(new_lens=i32([1, 2])), dict(status=i32([0, 0])), dict(workspace=one)):
        kw = dict(rows=one, new_lens=one, block_size=16)
        with pytest.raises(ValueError):
            mr.pages_grow(*d.state, **{**kw, **bad})
    with pytest.raises(mr.MropeError):
        mr.pages_grow(*d.state, i32([0] * 5), i32([1] * 5), 16)
    with pytest.raises(mr.MropeError):
        mr.pages_grow(*d.state, one, one, 0)
    with pytest.raises(ValueError):
        mr.pages_fork(*d.state, one, one, 16, [torch.zeros(7, 4, device="cuda")])
    with pytest.raises(ValueError):
        mr.pages_compact(*d.state, [torch.zeros(8, 4, 4, device="cuda").transpose(1, 2)])
    with pytest.raises(ValueError):
        mr.pages_compact(d.refcount, d.tables.long(), d.lens, d.pools)
    with pytest.raises(ValueError):
        mr.pages_copy(one, one, [])
    d.check()


def test_pages_graph():
    """Grow and fork captured once: replays on a restored state give what the eager calls gave."""
    d = Dev(200, 12, 20, 16, 6)
    rows, lens = i32([0, 1, 2]), i32([100, 33, 64])
    src, dst = i32([0, 1, 0]), i32([5, 6, 7])
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    st = i32([0, 0, 0])
    save = [x.clone() for x in (*d.state, *d.pools)]

    def run():
        mr.pages_grow(*d.state, rows, lens, 16, status=st, workspace=ws)
        mr.pages_fork(*d.state, src, dst, 16, d.pools, status=st, workspace=ws)

    run()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*d.state, *d.pools, st)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(4):
        for a, b in zip((*d.state, *d.pools), save):
            a.copy_(b)
        ws.fill_(i)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip((*d.state, *d.pools, st), want)), i
        torch.ones(1 << 20, device="cuda").sum().item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_serving_loop(dtype):
    """As a server uses them: prompts get pages, planes come from ids, the append and the attention run,
    rows generate, one is forked and both go on, one leaves, the pool is compacted, and the rest go on --
    every output against 64 bits on the codes that the cache holds, and the codes against the reference."""
    bs, hq, hk, D, n_rows, n_pages = 16, 8, 2, 256, 6, 60
    g = torch.Generator().manual_seed(21)
    d = Dev(n_pages, n_rows, 12, bs, 7)
    kc, vc = (torch.zeros(n_pages, bs, hk, D, device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.ones(n_pages, hk, device="cuda") for _ in range(2))
    cache = (kc, vc, ks, vs)
    host = [torch.zeros(n_pages, bs, hk, D).to(F8), torch.zeros(n_pages, bs, hk, D).to(F8), torch.ones(n_pages, hk), torch.ones(n_pages, hk)]
    pools = [kc.view(torch.uint8), vc.view(torch.uint8), ks, vs]
    hpools = [host[0].view(torch.uint8), host[1].view(torch.uint8), host[2], host[3]]
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    kept = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -20}[dtype]

    def heads(T, h):
        return torch.randn(T, h, D, generator=g).to(dtype)

    def attend(q, cu, rows, what):
        ctx, tab = d.lens[i32(rows).long()].contiguous(), d.tables[i32(rows).long()].contiguous()
        out, lse = mr.attend_kv8(q, cu, ctx, tab, *cache, return_lse=True)
        o, z, spread, amp = ref.attend(q.cpu(), None if cu is None else cu.tolist(), ctx.tolist(), tab.tolist(), *host)
        tol = half * 1.01 * o.abs() + (4 * D * 2.0 ** -24 * 2 * amp[..., None] + 2 * kept * (amp[..., None] if dtype == torch.float32 else 0)
                                       + kept + 2.0 ** -19) * spread + 1e-30
        assert bool(((out.cpu().double() - o).abs() <= tol).all()), what
        assert all(torch.equal(a.cpu(), b) for a, b in zip(pools, hpools)), what

    def generate(rows, amount, what):
        lens = [d.m.len[r] + 1 for r in rows]
        assert mr.pages_grow(*d.state, i32(rows), i32(lens), bs).tolist() == d.m.grow(rows, lens)
        q, k, v = heads(len(rows), hq), heads(len(rows), hk), heads(len(rows), hk)
        pos = [n - 1 for n in lens]
        tab = d.tables[i32(rows).long()].contiguous()
        qd = q.cuda()
        mr.decode_kv8(qd, k.cuda(), v.cuda(), i32(pos), i32([amount[r] for r in rows]), tab, *cache)
        planes = torch.tensor([p - amount[r] for p, r in zip(pos, rows)], dtype=torch.int32).expand(3, len(rows))
        kr = ref.rotate(k, planes)
        for i, r in enumerate(rows):
            ref.append(kr[i:i + 1], host[0], host[2], d.m.tab[r], pos[i])
            ref.append(v[i:i + 1].float(), host[1], host[3], d.m.tab[r], pos[i])
        attend(qd, None, rows, what)

    # prompts: an image prompt of 110 tokens, text of 45, 16 and 1
    rows, lens = [0, 1, 2, 3], [110, 45, 16, 1]
    assert mr.pages_grow(*d.state, i32(rows), i32(lens), bs).tolist() == d.m.grow(rows, lens) == [0] * 4
    ids = torch.randint(0, 1000, (sum(lens),), generator=g, dtype=torch.int32)
    ids[6] = mr.IMAGE_ID
    cu = i32([0, 110, 155, 171, 172])
    planes, _, amount, _, _ = mr.planes(ids.cuda(), cu)
    am = amount.tolist() + [0, 0]
    q, k, v = heads(172, hq), heads(172, hk), heads(172, hk)
    qd = q.cuda()
    tab = d.tables[:4].contiguous()
    mr.apply_kv8(qd, k.cuda(), v.cuda(), planes, cu, tab, *cache)
    kr = ref.rotate(k, planes.cpu())
    for r in rows:
        lo, hi = int(cu[r]), int(cu[r + 1])
        ref.append(kr[lo:hi], host[0], host[2], d.m.tab[r], 0)
        ref.append(v[lo:hi].float(), host[1], host[3], d.m.tab[r], 0)
    attend(qd, cu, rows, "prompts")
    for i in range(3):
        generate([0, 1, 2, 3], am, ("generate", i))
    say("fork")
    assert mr.pages_fork(*d.state, i32([0, 0]), i32([4, 5]), bs, pools).tolist() == d.m.fork([0, 0], [4, 5], hpools) == [0, 0]
    am[4] = am[5] = am[0]
    for i in range(2):
        generate([4, 0, 2, 5], am, ("forked", i))
    mr.pages_free(*d.state, i32([1, 0]))
    d.m.free([1, 0])
    assert mr.pages_compact(*d.state, pools).item() == d.m.compact(hpools)
    d.check("compact")
    for i in range(2):
        generate([5, 2, 3, 4], am, ("compacted", i))
    d.check("end")
