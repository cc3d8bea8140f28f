"""CPU checks of the C entry points and the binding for trees of drafted tokens: bad arguments are refused on the host
with the documented status, nothing is launched; and the plain forms that the GPU tests compare with are
themselves checked on cases worked out by hand."""
import ctypes
import math

import numpy as np
import pytest
import torch

import canvas_rope_rotary_amd as mr
import kv8_ref
import tree_ref as ref
from canvas_rope_rotary_amd import _lib

OK, ARG, ALIGN, UNSUP, WS, HIP = range(6)
BF16, F32 = _lib.MROPE_BF16, _lib.MROPE_F32
A = 1 << 20  # an aligned fake device address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


BASE = dict(par=A, n=100, cu=A, ns=4, pos=A, am=None, planes=A, ps=100, mask=A, mw=2,
            q=A, qt=2048, qh=256, nq=8, nk=2, hd=256, dt=BF16, ctx=A, tab=A, ts=8, tw=8, kc=A, vc=A, ks=A, vs=A, bs=16, nb=64,
            cb=8192, ct=512, ch=256, sc=0.0625, out=1 << 30, ot=2048, oh=256, lse=None, ws=A, wsb=1 << 40,
            t=A, tst=5000, d=None, dst=0, v=5000, ids=A, ua=A, un=A, nkept=A, path=A, nxt=A, nl=2)


def _planes(lib, **kw):
    a = {**BASE, **kw}
    return lib.mrope_planes_tree(a["par"], a["n"], a["cu"], a["ns"], a["pos"], a["am"], a["planes"], a["ps"], a["mask"], a["mw"], None)


def _attend(lib, **kw):
    a = {**BASE, **kw}
    return lib.mrope_attend_tree_kv8(a["q"], a["qt"], a["qh"], a["nq"], a["n"], a["nk"], a["hd"], a["dt"], a["cu"], a["ns"], a["ctx"],
                                     a["mask"], a["mw"], a["tab"], a["ts"], a["tw"], a["kc"], a["vc"], a["ks"], a["vs"], a["bs"],
                                     a["nb"], a["cb"], a["ct"], a["ch"], a["sc"], a["out"], a["ot"], a["oh"], a["lse"], a["ws"],
                                     a["wsb"], None)


def _verify(lib, **kw):
    a = {**BASE, **kw}
    return lib.mrope_verify_tree(a["t"], a["tst"], a["d"], a["dst"], a["v"], a["dt"], a["n"], a["ids"], a["par"], a["cu"], a["ns"],
                                 a["ua"], a["un"], a["nkept"], a["path"], a["nxt"], a["ws"], a["wsb"], None)


def _keep(lib, layers=True, **kw):
    a = {**BASE, **kw}
    arr = (ctypes.c_uint64 * (4 * 65))(*([a["kc"] or 0, a["vc"] or 0, a["ks"] or 0, a["vs"] or 0] * 65))
    return lib.mrope_keep_kv8(arr if layers else None, a["nl"], a["nk"], a["hd"], a["bs"], a["nb"], a["cb"], a["ct"], a["ch"], a["nkept"],
                              a["path"], a["n"], a["cu"], a["ns"], a["pos"], a["tab"], a["ts"], a["tw"], None)


TREES = [(dict(n=-1), ARG), (dict(n=(1 << 31) - 1, ps=1 << 31), ARG), (dict(ns=-1), ARG), (dict(ns=0), ARG), (dict(cu=None), ARG), (dict(cu=A + 2), ALIGN)]
CACHE = [(dict(bs=8), UNSUP), (dict(bs=128), UNSUP), (dict(hd=96, qh=96, ct=512), UNSUP), (dict(nk=0), UNSUP), (dict(nk=65), UNSUP),
         (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(ks=None), ARG), (dict(vs=None), ARG), (dict(tab=None), ARG), (dict(nb=-1), ARG),
         (dict(tw=-1), ARG), (dict(ts=7), ARG), (dict(ct=128), ARG), (dict(ch=128), ARG), (dict(kc=A + 8), ALIGN), (dict(vc=A + 4), ALIGN),
         (dict(ct=520), ALIGN), (dict(cb=8200), ALIGN), (dict(ks=A + 2), ALIGN), (dict(tab=A + 1), ALIGN)]


@pytest.mark.parametrize("kw,code", TREES + [
    (dict(mw=0), ARG), (dict(mw=17), ARG), (dict(ps=99), ARG), (dict(par=None), ARG), (dict(pos=None), ARG), (dict(planes=None), ARG),
    (dict(mask=None), ARG), (dict(mask=A + 4), ALIGN), (dict(par=A + 1), ALIGN), (dict(am=A + 2), ALIGN), (dict(ns=1 << 25), ARG)])
def test_planes_tree_refusals(lib, kw, code):
    assert _planes(lib, **kw) == code
    assert lib.mrope_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", TREES + CACHE + [
    (dict(mw=0), ARG), (dict(mw=65), ARG), (dict(mask=None), ARG), (dict(mask=A + 4), ALIGN), (dict(nq=7), UNSUP), (dict(nq=0), UNSUP),
    (dict(nq=65), UNSUP), (dict(dt=9), UNSUP), (dict(out=None), ARG), (dict(out=A), ARG), (dict(out=A + 8), ALIGN), (dict(oh=128), ARG),
    (dict(q=None), ARG), (dict(qt=2044), ALIGN), (dict(ctx=None), ARG), (dict(sc=float("nan")), ARG), (dict(sc=1e300), ARG),
    (dict(lse=A + 2), ALIGN), (dict(ws=None, tw=1 << 12, ts=1 << 12), WS), (dict(ws=A + 16, tw=1 << 12, ts=1 << 12), WS),
    (dict(wsb=16, tw=1 << 12, ts=1 << 12), WS), (dict(tw=1 << 24, ts=1 << 24), ARG), (dict(n=1 << 28), ARG)])
def test_attend_tree_refusals(lib, kw, code):
    assert _attend(lib, **kw) == code


@pytest.mark.parametrize("kw,code", TREES + [
    (dict(dt=9), UNSUP), (dict(v=0), ARG), (dict(v=-5), ARG), (dict(tst=4999), ARG), (dict(d=A, dst=4999), ARG), (dict(t=A + 1), ALIGN),
    (dict(d=A + 1, dst=5000), ALIGN), (dict(t=A + 2, dt=F32), ALIGN), (dict(ids=A + 2), ALIGN), (dict(nkept=A + 1), ALIGN), (dict(t=None), ARG),
    (dict(ids=None), ARG), (dict(ua=None), ARG), (dict(un=None), ARG), (dict(nkept=None), ARG), (dict(path=None), ARG), (dict(nxt=None), ARG),
    (dict(ws=None), WS), (dict(ws=A + 8), WS), (dict(wsb=64), WS), (dict(ns=1 << 24), ARG)])
def test_verify_tree_refusals(lib, kw, code):
    assert _verify(lib, **kw) == code


@pytest.mark.parametrize("kw,code", TREES + CACHE + [
    (dict(nl=-1), ARG), (dict(nl=65), ARG), (dict(layers=False), ARG), (dict(nkept=None), ARG), (dict(path=None), ARG), (dict(pos=None), ARG),
    (dict(path=A + 2), ALIGN), (dict(cb=4096), ARG), (dict(ch=512), ARG), (dict(ns=1 << 28), ARG)])
def test_keep_refusals(lib, kw, code):
    assert _keep(lib, **kw) == code


def test_nothing_to_do(lib):
    assert _planes(lib, n=0, ns=0, cu=None) == OK and _planes(lib, n=0) == OK
    assert _attend(lib, n=0, ns=0) == OK
    assert _verify(lib, n=0, ns=0, cu=None) == OK
    assert _keep(lib, n=0, ns=0) == OK and _keep(lib, nl=0) == OK


def test_workspace_bytes(lib):
    f = lib.mrope_attend_tree_kv8_workspace_bytes
    assert f(0, 4, 8, 2, 256, BF16, 8, 16) == 0
    assert f(4, 4, 8, 3, 256, BF16, 8, 16) == 0   # refused shapes need none
    assert f(4, 4, 8, 2, 256, BF16, 0, 16) == 0   # an empty table holds nothing
    assert f(4, 4, 8, 2, 256, BF16, 8, 16) == 0   # one chunk: nothing to join
    assert 0 < f(32, 1, 8, 2, 256, BF16, 1 << 20, 16) <= 1 << 27  # bounded however long the table
    g = lib.mrope_verify_tree_workspace_bytes
    assert g(0, 5000, 1, 1) == 0 and g(4, 0, 1, 1) == 0
    assert g(4, 5000, 0, 1) == g(4, 5000, 1, 0) > 0          # nothing to sum on the way
    assert g(4, 5000, 1, 1) > g(4, 5000, 0, 1)


def test_binding_refuses_the_cpu():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mr.planes_tree(i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        mr.verify_tree(torch.zeros(3, 5), i, None, i, torch.zeros(3), torch.zeros(2))
    with pytest.raises(ValueError):
        mr.keep_kv8(i, i, i, i, i, [])


# ---------------------------------------------------------------- the plain forms ---------------
def test_planes_by_hand():
    #      0 - 1 - 3      and a second sequence with a root of its own in the middle
    #       \- 2 - 4 - 5
    parents = [-1, 0, 0, 1, 2, 4, 9, 0, -1, 2]
    planes, mask = ref.planes_tree(parents, [0, 6, 10], [100, 7], [58, 0], 1)
    assert planes[0].tolist() == [42, 43, 43, 44, 44, 45, 7, 8, 7, 8]
    assert planes[1].tolist() == planes[2].tolist() == planes[0].tolist()
    assert mask[:, 0].tolist() == [1, 3, 5, 11, 21, 53, 1, 3, 4, 12]


def test_verify_by_hand():
    p = np.array([[0.5, 0.3, 0.2, 0.0], [0.0, 0.0, 0.25, 0.75], [0.1, 0.2, 0.3, 0.4]])
    # children 1 (id 1) and 2 (id 0) of token 0: u * 1 < 0.3, then u * 0.7 < 0.5
    one = lambda u1, u2, un: ref.verify_one(p, [9, 1, 0], [-1, 0, 0], [0, u1, u2], un)
    assert one(0.29, 0.0, 0.3) == ([0, 1], 3)
    assert one(0.3, 0.71, 0.2) == ([0, 2], 1)
    assert one(0.3, 0.72, 0.99) == ([0], 2)      # what is left: only token 2
    # drawn: r = max(p - q, 0) = (.25, 0, .2, 0) with Z = .45 after the first refusal, which leaves the second child's
    # token nothing; then r = (.1375, 0, .2, 0)
    q = np.array([[0.25, 0.75, 0.0, 0.0]] * 3)
    assert ref.verify_one(p, [9, 1, 1], [-1, 0, 0], [0, 0.41, 0.0], 0.4, q) == ([0], 0)
    assert ref.verify_one(p, [9, 1, 1], [-1, 0, 0], [0, 0.41, 0.0], 0.41, q) == ([0], 2)
    assert ref.verify_one(p, [9, 1, 1], [-1, 0, 0], [0, 0.39, 0.0], 0.0, q) == ([0, 1], 2)


def test_drawn_drafts_keep_the_targets_distribution():
    """The first token after the walk's first step is distributed as the target, whatever the drafter: summed over
    all draws of two siblings and the random numbers, exactly."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    got = np.zeros(3)
    for a in range(3):
        for b in range(3):
            pr = q[a] * q[b]
            keep_a = min(1.0, p[a] / q[a])
            got[a] += pr * keep_a
            r = np.maximum(p - q, 0)
            z = r.sum()
            keep_b = min(1.0, r[b] / (q[b] * z))
            got[b] += pr * (1 - keep_a) * keep_b
            r2 = np.maximum(p - (1 + z) * q, 0)
            assert np.allclose(r2, np.maximum(r - z * q, 0))
            got += pr * (1 - keep_a) * (1 - keep_b) * (r2 / r2.sum() if r2.sum() > 0 else p)
    assert np.allclose(got, p)


def test_keep_by_hand():
    F8 = torch.float8_e4m3fn
    cache = torch.zeros(3, 16, 1, 64).to(F8)
    scale = torch.tensor([[1.0], [4.0], [0.5]])
    cache[1, 14] = torch.full((1, 64), 8.0).to(F8)   # position 14: 32
    cache[1, 15] = torch.full((1, 64), 448.0).to(F8)  # position 15: 1792
    cache[2, 1] = torch.full((1, 64), 3.0).to(F8)    # position 17: 1.5
    cache[2, 3] = torch.full((1, 64), 256.0).to(F8)  # position 19: 128
    ref.keep([3], [0, 2, 4, -1, -1], [0, 5], [15], [[1, 2]], cache, scale)
    assert scale.flatten().tolist() == [1.0, 4.0, 0.5]  # 128 needs 2^-1 (224 * 2^-1 = 112 < 128 <= 448 * 2^-1)
    assert cache[1, 15, 0, 0] == 448.0 and cache[2, 0, 0, 0] == 3.0 and cache[2, 1, 0, 0] == 256.0
    ref.keep([2], [0, 2, -1, -1, -1], [0, 5], [15], [[1, 2]], cache, scale)  # page 2 then holds position 17's 128, at 16
    assert float(scale[2]) == 0.5 and cache[2, 0, 0, 0] == 256.0
    assert kv8_ref.scale_exp(128.0) == -1 and math.log2(0.5) == -1
