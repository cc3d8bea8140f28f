"""What the calls for trees of drafted tokens refuse to write, through the binding: memory that they would write twice, or read
and write at once."""
import pytest
import torch

import canvas_rope_rotary_amd as mr
from test_gpu_kv8 import World, bits, i32

pytestmark = pytest.mark.gpu


def test_keep_refuses_a_cache_twice():
    """The same cache for two layers, K in V's place, a layer that begins within another: refused, and nothing is moved."""
    w = World([60], 16, 2, 128, seed=81)
    kc, vc, ks, vs = w.cache()
    k2, v2, ks2, vs2 = w.cache()
    args = (i32([3]).cuda(), i32([0, 2, 4, -1, -1, -1]).cuda(), i32([0, 6]).cuda(), i32([40]).cuda(), w.tables.cuda())
    wide = torch.zeros(w.nb + 1, *kc.shape[1:], dtype=torch.uint8, device="cuda")
    for caches in ([(kc, vc, ks, vs)] * 2, [(kc, kc, ks, vs)], [(kc, vc, ks, ks)], [(kc, vc, ks, vs), (k2, vc, ks2, vs2)],
                   [(kc, vc, ks, vs), (k2, v2, ks2, vs)], [(wide[1:], wide[:-1], ks, vs)]):
        with pytest.raises(mr.MropeError, match="share"):
            mr.keep_kv8(*args, caches)
    assert torch.equal(bits(kc), bits(w.kc)) and torch.equal(bits(vc), bits(w.vc)) and torch.equal(ks.cpu(), w.ks)
    mr.keep_kv8(*args, [(kc, vc, ks, vs), (k2, v2, ks2, vs2)])
    assert torch.equal(bits(kc), bits(k2)) and torch.equal(bits(vc), bits(v2)) and not torch.equal(bits(kc), bits(w.kc))


def test_verify_refuses_its_inputs_place():
    """Path, counts and next tokens in the place of an input or of one another: refused.  Beside them, and between the rows of
    distributions: the same results as anywhere."""
    g = torch.Generator().manual_seed(82)
    T, vocab = 9, 501
    room = torch.zeros(T, vocab + 11, device="cuda")
    target = room[:, :vocab]
    target.copy_(torch.softmax(torch.randn(T, vocab, generator=g) * 4, 1))
    flat = torch.zeros(60, dtype=torch.int32, device="cuda")
    ids, parents, cu = flat[:9], flat[9:18], flat[18:21]
    ids.copy_(i32([0] + target[0].argsort(descending=True)[:8].tolist()))
    parents.copy_(i32([-1, 0, 0, 1, 1, -1, 0, 0, 0]))
    cu.copy_(i32([0, 5, 9]))
    u, un = torch.rand(T, generator=g).cuda(), torch.rand(2, generator=g).cuda()
    want = [x.tolist() for x in mr.verify_tree(target, ids.clone(), parents.clone(), cu.clone(), u, un)]
    two = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(path=ids), dict(path=parents), dict(path=flat[20:29]), dict(path=u.view(torch.int32)), dict(n_kept=cu[:2]),
               dict(n_kept=ids[3:5]), dict(next_ids=un.view(torch.int32)), dict(n_kept=two, next_ids=two),
               dict(n_kept=room.view(torch.int32)[3, 4:6]), dict(next_ids=room.view(torch.int32)[8, vocab - 1:vocab + 1])):
        with pytest.raises(mr.MropeError, match="overlap"):
            mr.verify_tree(target, ids, parents, cu, u, un, **kw)
    gap = room.view(torch.int32)
    got = mr.verify_tree(target, ids, parents, cu, u, un, path=flat[21:30], n_kept=gap[2, vocab:vocab + 2], next_ids=gap[8, vocab + 9:])
    assert [x.tolist() for x in got] == want and ids.tolist()[0] == 0 and cu.tolist() == [0, 5, 9]


def test_planes_refuse_their_inputs_place():
    flat = torch.zeros(80, dtype=torch.int32, device="cuda")
    parents, cu, pos = flat[:6], flat[6:9], flat[10:12]
    parents.copy_(i32([-1, 0, 0, -1, 0, 1]))
    cu.copy_(i32([0, 3, 6]))
    pos.copy_(i32([50, 70]))
    want = [x.tolist() for x in mr.planes_tree(parents, cu, pos)]
    for kw in (dict(planes=flat[:18].view(3, 6)), dict(planes=flat[5:23].view(3, 6)), dict(mask=flat[:12].view(torch.int64).view(6, 1)),
               dict(planes=flat[20:38].view(3, 6), mask=flat[36:48].view(torch.int64).view(6, 1))):
        with pytest.raises(mr.MropeError, match="overlap"):
            mr.planes_tree(parents, cu, pos, **kw)
    got = mr.planes_tree(parents, cu, pos, planes=flat[12:30].view(3, 6), mask=flat[30:42].view(torch.int64).view(6, 1))
    assert [x.tolist() for x in got] == want
    planes = torch.as_strided(flat, (3, 6), (20, 1), 20)
    mask = torch.as_strided(flat, (12,), (1,), 28).view(torch.int64).view(6, 1)  # between the first two rows
    got = mr.planes_tree(parents, cu, pos, planes=planes, mask=mask)
    assert [x.tolist() for x in got] == want


def test_attend_refuses_its_inputs_place():
    """Outputs in the place of the mask, the lengths or one another: refused.  Log-sums in the gap between two rows of queries: the
    same as anywhere."""
    w = World([40], 16, 2, 128, seed=83)
    room = torch.zeros(7, 9, 128, device="cuda")
    q = room[:, :8]
    q.copy_(w.heads(7, 8, "f32"))
    cu, ctx, tab, cache = i32([0, 7]).cuda(), i32([40]).cuda(), w.tables.cuda(), w.cache()
    mask = torch.full((7, 28), -1, dtype=torch.int64, device="cuda")
    out, lse = mr.attend_tree_kv8(q, cu, ctx, mask, tab, *cache, return_lse=True)
    for bad in (mask.view(torch.float32).view(-1)[:56].view(7, 8), room[3, 7][:56].view(7, 8)):
        with pytest.raises(mr.MropeError, match="overlap"):
            mr.attend_tree_kv8(q, cu, ctx, mask, tab, *cache, lse=bad)
    big = torch.zeros(7 * 8 * 128 + 64, device="cuda")
    with pytest.raises(mr.MropeError, match="overlap"):
        mr.attend_tree_kv8(q, cu, ctx, mask, tab, *cache, out=big[:7168].view(7, 8, 128), lse=big[7120:7176].view(7, 8))
    with pytest.raises(mr.MropeError, match="overlap"):
        mr.attend_tree_kv8(q, cu, ctx, big[6000:6014].view(torch.int64).view(7, 1), tab, *cache, out=big[:7168].view(7, 8, 128))
    gap = room[2, 8][:56].view(7, 8)
    o2, z2 = mr.attend_tree_kv8(q, cu, ctx, mask, tab, *cache, lse=gap)
    assert z2 is gap and torch.equal(o2, out) and torch.equal(z2, lse)
