"""CPU checks of the 8-bit cache's and the page calls' C entry points: bad arguments are refused on the
host with the documented status.  No call here passes validation with work to do, so nothing is launched."""
import ctypes

import pytest

from canvas_rope_rotary_amd import _lib
from canvas_rope_rotary_amd._lib import MropePool

OK, ARG, ALIGN, UNSUP, WS, HIP = range(6)
BF16, F32 = _lib.MROPE_BF16, _lib.MROPE_F32
A = 1 << 20  # an aligned fake device address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


BASE = dict(q=A, qt=2048, qh=256, nq=8, k=A, kt=512, kh=256, nk=2, v=A, vt=512, vh=256, n=100, hd=256, rot=64, dt=BF16,
            planes=A, ps=100, theta=1e7, cu=A, ns=4, off=None, tab=A, ts=8, tw=8, kc=A, vc=A, ks=A, vs=A, bs=16, nb=64,
            cb=8192, ct=512, ch=256, pos=A, am=A)


def _apply(lib, **kw):
    a = {**BASE, **kw}
    return lib.mrope_apply_kv8(a["q"], a["qt"], a["qh"], a["nq"], a["k"], a["kt"], a["kh"], a["nk"], a["v"], a["vt"], a["vh"],
                               a["n"], a["hd"], a["rot"], a["dt"], a["planes"], a["ps"], a["theta"], a["cu"], a["ns"], a["off"],
                               a["tab"], a["ts"], a["tw"], a["kc"], a["vc"], a["ks"], a["vs"], a["bs"], a["nb"], a["cb"], a["ct"],
                               a["ch"], None)


def _decode(lib, **kw):
    a = {**BASE, **kw}
    return lib.mrope_decode_kv8(a["q"], a["qt"], a["qh"], a["nq"], a["k"], a["kt"], a["kh"], a["nk"], a["v"], a["vt"], a["vh"],
                                a["ns"], a["pos"], a["am"], a["tab"], a["ts"], a["tw"], a["kc"], a["vc"], a["ks"], a["vs"],
                                a["bs"], a["nb"], a["cb"], a["ct"], a["ch"], a["hd"], a["rot"], a["dt"], a["theta"], None)


def _attend(lib, **kw):
    a = {**BASE, **dict(ctx=A, out=A, ot=2048, oh=256, lse=None, ws=A, wsb=1 << 40, sc=0.0625), **kw}
    return lib.mrope_attend_kv8(a["q"], a["qt"], a["qh"], a["nq"], a["n"], a["nk"], a["hd"], a["dt"], a["cu"], a["ns"], a["ctx"],
                                a["tab"], a["ts"], a["tw"], a["kc"], a["vc"], a["ks"], a["vs"], a["bs"], a["nb"], a["cb"], a["ct"],
                                a["ch"], a["sc"], a["out"], a["ot"], a["oh"], a["lse"], a["ws"], a["wsb"], None)


CACHE_CASES = [
    (dict(bs=8), UNSUP), (dict(bs=48), UNSUP), (dict(bs=128), UNSUP), (dict(hd=96, qh=96, kh=96, vh=96), UNSUP),
    (dict(nk=0), UNSUP), (dict(nk=65), UNSUP), (dict(dt=9), UNSUP),
    (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(ks=None), ARG), (dict(vs=None), ARG), (dict(tab=None), ARG),
    (dict(nb=-1), ARG), (dict(nb=1 << 31), ARG), (dict(tw=-1), ARG), (dict(ts=7), ARG), (dict(ct=128), ARG), (dict(ch=128), ARG),
    (dict(cb=-16), ARG), (dict(kc=A + 8), ALIGN), (dict(vc=A + 4), ALIGN), (dict(ct=520), ALIGN), (dict(cb=8200), ALIGN),
    (dict(ks=A + 2), ALIGN), (dict(tab=A + 1), ALIGN), (dict(q=A + 8), ALIGN), (dict(qt=2044), ALIGN), (dict(ns=-1), ARG),
]


@pytest.mark.parametrize("kw,code", CACHE_CASES + [
    (dict(v=None), ARG), (dict(q=None), ARG), (dict(k=None), ARG), (dict(planes=None), ARG), (dict(ps=99), ARG), (dict(cu=None), ARG),
    (dict(ns=0), ARG), (dict(theta=0.0), ARG), (dict(rot=32), UNSUP), (dict(v=A + 8), ALIGN), (dict(vh=252), ARG), (dict(vt=500), ALIGN),
    (dict(nq=65), UNSUP), (dict(n=-1), ARG), (dict(n=1 << 29, ps=1 << 29), ARG),
])
def test_apply_kv8_refusals(lib, kw, code):
    assert _apply(lib, **kw) == code
    assert lib.mrope_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", CACHE_CASES + [
    (dict(v=None), ARG), (dict(pos=None), ARG), (dict(am=None), ARG), (dict(theta=float("inf")), ARG), (dict(ns=1 << 28), ARG),
])
def test_decode_kv8_refusals(lib, kw, code):
    assert _decode(lib, **kw) == code


@pytest.mark.parametrize("kw,code", CACHE_CASES + [
    (dict(nq=7), UNSUP), (dict(nq=0), UNSUP), (dict(nq=65), UNSUP), (dict(out=None), ARG), (dict(out=A + 8), ALIGN), (dict(oh=128), ARG),
    (dict(ctx=None), ARG), (dict(cu=None), ARG), (dict(ns=0), ARG), (dict(sc=float("nan")), ARG), (dict(sc=float("inf")), ARG),
    (dict(lse=A + 2), ALIGN), (dict(ws=None, tw=1 << 12, ts=1 << 12), WS), (dict(ws=A + 16, tw=1 << 12, ts=1 << 12), WS),
    (dict(wsb=16, tw=1 << 12, ts=1 << 12), WS), (dict(tw=1 << 24, ts=1 << 24), ARG), (dict(n=1 << 28), ARG),
])
def test_attend_kv8_refusals(lib, kw, code):
    assert _attend(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(out=A), ARG), (dict(out=2 * A, sc=1e300), ARG), (dict(out=2 * A, sc=-3e38), ARG), (dict(out=2 * A, ws=None, tw=1 << 12, ts=1 << 12), WS),
    (dict(out=2 * A, n=100, ns=1 << 19, nq=64, nk=64, kh=256, ct=1 << 14, qt=1 << 14, ot=1 << 14), ARG),
])
def test_attend_kv8_refusals_in_place_and_out_of_range(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_kv8_nothing_to_do(lib):
    assert _apply(lib, n=0, ns=0, cu=None, planes=None) == OK
    assert _decode(lib, ns=0) == OK
    assert _attend(lib, n=0, ns=0) == OK


def test_attend_workspace_bytes(lib):
    f = lib.mrope_attend_kv8_workspace_bytes
    assert f(0, 4, 8, 2, 256, BF16, 0, 8, 16) == 0
    assert f(4, 4, 8, 3, 256, BF16, 1, 8, 16) == 0     # refused shapes need none
    assert f(4, 4, 8, 2, 256, BF16, 1, 0, 16) == 0     # an empty table holds nothing
    one = f(1, 1, 8, 2, 256, BF16, 1, 2048, 16)
    assert one > 0
    # bounded however long the table: a fixed number of partial results, each of 8 rows
    assert f(1, 1, 8, 2, 256, BF16, 1, 1 << 20, 16) <= 1 << 27


STATE = dict(ref=A, nb=64, tab=A, ts=8, tw=8, lens=A, nr=16, bs=16, rows=A, new=A, n=4, st=A, ws=A, wsb=1 << 30)


def _pools(n=2, **kw):
    a = (MropePool * max(1, n))()
    for p in a:
        p.ptr, p.page_bytes, p.page_stride = kw.get("ptr", A), kw.get("bytes", 8192), kw.get("stride", 8192)
    return a


def _grow(lib, **kw):
    a = {**STATE, **kw}
    return lib.mrope_pages_grow(a["ref"], a["nb"], a["tab"], a["ts"], a["tw"], a["lens"], a["nr"], a["bs"], a["rows"], a["new"], a["n"],
                                a["st"], a["ws"], a["wsb"], None)


def _free(lib, **kw):
    a = {**STATE, **kw}
    return lib.mrope_pages_free(a["ref"], a["nb"], a["tab"], a["ts"], a["tw"], a["lens"], a["nr"], a["rows"], a["n"], None)


def _fork(lib, pools=None, np_=2, **kw):
    a = {**STATE, **kw}
    return lib.mrope_pages_fork(a["ref"], a["nb"], a["tab"], a["ts"], a["tw"], a["lens"], a["nr"], a["bs"], a["rows"], a["new"], a["n"],
                                a["st"], _pools() if pools is None else pools, np_, a["ws"], a["wsb"], None)


def _compact(lib, pools=None, np_=2, moved=A, **kw):
    a = {**STATE, **kw}
    return lib.mrope_pages_compact(a["ref"], a["nb"], a["tab"], a["ts"], a["tw"], a["lens"], a["nr"], moved,
                                   _pools() if pools is None else pools, np_, a["ws"], a["wsb"], None)


STATE_CASES = [(dict(ref=None), ARG), (dict(tab=None), ARG), (dict(lens=None), ARG), (dict(nb=-1), ARG), (dict(nb=(1 << 24) + 1), ARG),
               (dict(nr=-1), ARG), (dict(nr=(1 << 22) + 1), ARG), (dict(ts=7), ARG), (dict(tw=-1), ARG), (dict(ref=A + 2), ALIGN),
               (dict(lens=A + 1), ALIGN)]
WS_CASES = [(dict(ws=None), WS), (dict(ws=A + 4), WS), (dict(wsb=64), WS)]


@pytest.mark.parametrize("kw,code", STATE_CASES + WS_CASES + [(dict(bs=0), ARG), (dict(n=17), ARG), (dict(n=-1), ARG), (dict(rows=None), ARG),
                                                              (dict(new=None), ARG), (dict(st=None), ARG)])
def test_pages_grow_refusals(lib, kw, code):
    assert _grow(lib, **kw) == code


@pytest.mark.parametrize("kw,code", STATE_CASES + [(dict(rows=None), ARG), (dict(n=17), ARG)])
def test_pages_free_refusals(lib, kw, code):
    assert _free(lib, **kw) == code


@pytest.mark.parametrize("kw,code", STATE_CASES + WS_CASES + [
    (dict(bs=-1), ARG), (dict(rows=None), ARG), (dict(np_=65), ARG), (dict(np_=-1), ARG), (dict(pools=_pools(ptr=None)), ARG),
    (dict(pools=_pools(bytes=0)), ARG), (dict(pools=_pools(stride=100)), ARG)])
def test_pages_fork_refusals(lib, kw, code):
    assert _fork(lib, **kw) == code


@pytest.mark.parametrize("kw,code", STATE_CASES + WS_CASES + [(dict(moved=None), ARG), (dict(np_=65), ARG), (dict(pools=_pools(bytes=-4)), ARG)])
def test_pages_compact_refusals(lib, kw, code):
    assert _compact(lib, **kw) == code


def test_pages_copy_refusals(lib):
    f = lib.mrope_pages_copy
    assert f(_pools(), 2, 64, None, A, 4, None) == ARG
    assert f(_pools(), 2, 64, A, A, -1, None) == ARG
    assert f(_pools(), 65, 64, A, A, 4, None) == ARG
    assert f(_pools(), 2, -1, A, A, 4, None) == ARG
    assert f(_pools(), 2, 64, A, A, 0, None) == OK


def test_pages_nothing_to_do(lib):
    assert _grow(lib, n=0) == OK and _free(lib, n=0) == OK and _fork(lib, n=0) == OK


def test_pages_workspace_bytes(lib):
    r = lambda n: (n + 63) // 64 * 64
    for nb, nr in ((0, 0), (1, 1), (64, 16), (65, 1000), (1 << 20, 4096)):
        assert lib.mrope_pages_workspace_bytes(nb, nr) == 4 * (64 + 3 * r(nr) + 3 * r(nb))
