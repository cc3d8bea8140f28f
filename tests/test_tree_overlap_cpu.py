"""CPU checks of what the calls for trees of drafted tokens refuse to write: memory that they would write twice, or read and
write at once.  Nothing is launched."""
import ctypes
import itertools
import random

import pytest

from test_tree_abi_cpu import A, ARG, BASE, _attend, _planes, _verify, lib  # noqa: F401  (lib: a fixture)


# ---------------------------------------------------------------- keep --------------------------
def keep(lib, layers, **kw):  # noqa: F811
    """Status and message of a call whose last argument to be looked at, n_kept, is missing."""
    a = {**BASE, "nkept": None, **kw}
    flat = [p for layer in layers for p in layer]
    arr = (ctypes.c_uint64 * len(flat))(*flat)
    st = lib.mrope_keep_kv8(arr, len(layers), a["nk"], a["hd"], a["bs"], a["nb"], a["cb"], a["ct"], a["ch"], a["nkept"], a["path"], a["n"],
                            a["cu"], a["ns"], a["pos"], a["tab"], a["ts"], a["tw"], None)
    return st, lib.mrope_last_error().decode()


def apart(result):
    assert result[0] == ARG and ("share" in result[1] or "n_kept" in result[1]), result
    return "n_kept" in result[1]


CACHE, SCALE = 64 * 8192, 64 * 2 * 4  # bytes of a cache and its scales in BASE


def layers_of(n):
    return [[A + 2 * i * CACHE, A + (2 * i + 1) * CACHE, (1 << 40) + 2 * i * SCALE, (1 << 40) + (2 * i + 1) * SCALE] for i in range(n)]


@pytest.mark.parametrize("n", [1, 2, 6, 64])
def test_keep_takes_caches_side_by_side(lib, n):  # noqa: F811
    assert apart(keep(lib, layers_of(n)))


@pytest.mark.parametrize("n", [2, 64])
@pytest.mark.parametrize("what", [0, 1, 2, 3])
def test_keep_refuses_a_layer_twice(lib, n, what):  # noqa: F811
    layers = layers_of(n)
    layers[n - 1][what] = layers[0][what]
    assert not apart(keep(lib, layers))
    layers = layers_of(n)
    layers[n - 1][what ^ 1] = layers[0][what]  # K in V's place
    assert not apart(keep(lib, layers))


@pytest.mark.parametrize("what", [0, 2])
def test_keep_refuses_k_and_v_in_one(lib, what):  # noqa: F811
    layers = layers_of(1)
    layers[0][what + 1] = layers[0][what]
    assert not apart(keep(lib, layers))


@pytest.mark.parametrize("by,fine", [(CACHE, True), (CACHE - 16, False), (16, False), (8192, False)])
def test_keep_caches_that_overlap_in_part(lib, by, fine):  # noqa: F811
    layers = layers_of(1)
    layers[0][1] = layers[0][0] + by
    assert apart(keep(lib, layers)) is fine


@pytest.mark.parametrize("by,fine", [(SCALE, True), (SCALE - 4, False), (4, False)])
def test_keep_scales_that_overlap_in_part(lib, by, fine):  # noqa: F811
    layers = layers_of(1)
    layers[0][3] = layers[0][2] + by
    assert apart(keep(lib, layers)) is fine


def test_keep_empty_pool(lib):  # noqa: F811
    assert apart(keep(lib, [[0, 0, 0, 0]] * 2, nb=0))


def test_keep_layers_by_every_row(lib):  # noqa: F811
    """Two caches with their dimensions in any order and gaps, at every distance of some rows: refused exactly where a row of one
    touches a row of the other."""
    rng = random.Random(5)
    seen = [0, 0]
    for turn in range(400):
        nk, nb, bs, D = rng.randrange(1, 4), rng.randrange(1, 4), 16, 64
        strides, span = {}, D
        for name, extent in rng.sample([("ch", nk), ("ct", bs), ("cb", nb)], 3):
            strides[name] = max(-(-span // 16) * 16 + 16 * rng.choice([0, 0, 1, 5, 40]), D)
            if extent > 1:
                span += (extent - 1) * strides[name]
        d = 16 * rng.randrange(0, span // 16 + 3)
        rows = [b * strides["cb"] + t * strides["ct"] + h * strides["ch"] for b, t, h in itertools.product(range(nb), range(bs), range(nk))]
        taken = {r + x for r in rows for x in range(0, D, 16)}
        fine = not any(r + d + x in taken for r in rows for x in range(0, D, 16))
        pair = [A, A + d] if turn % 2 else [A + d, A]
        got = keep(lib, [[*pair, 1 << 40, 1 << 41]], nk=nk, nb=nb, bs=bs, hd=D, ts=8, **strides)
        assert apart(got) is fine, (nk, nb, strides, d)
        seen[fine] += 1
    assert min(seen) > 50


# ---------------------------------------------------------------- planes and verification -------
# 100 tokens of 4 sequences, each argument at a place of its own, 1 MB apart
PLACES = {name: A << 4 | i << 20 for i, name in enumerate(["par", "cu", "pos", "am", "planes", "mask", "ids", "ua", "un", "nkept", "path", "nxt"])}
FAR = dict(PLACES, t=1 << 40, d=1 << 41, dst=5000)
VECTORS = dict(par=400, cu=20, pos=16, am=16, ids=400, ua=400, un=16, nkept=16, path=400, nxt=16)  # bytes


def refused(st, message):
    return st == ARG and "overlap" in message


def planes(lib, **kw):  # noqa: F811
    return refused(_planes(lib, **{**PLACES, **kw}), lib.mrope_last_error().decode())


def verify(lib, **kw):  # noqa: F811
    return refused(_verify(lib, **{**FAR, **kw}), lib.mrope_last_error().decode())


@pytest.mark.parametrize("name", ["par", "cu", "pos", "am"])
@pytest.mark.parametrize("out,size", [("planes", 400), ("mask", 1600)])
def test_planes_over_its_inputs(lib, name, out, size):  # noqa: F811
    at, n = PLACES[name], VECTORS[name]
    assert planes(lib, **{out: at}) and planes(lib, **{out: at + (n - 4) // 8 * 8}) and planes(lib, **{out: at - size + 8})
    if out == "planes":  # its second and third rows
        assert planes(lib, planes=at - 4 * 5000, ps=5000) and planes(lib, planes=at - 8 * 5000 + n - 4, ps=5000)


def test_planes_over_its_mask(lib):  # noqa: F811
    assert planes(lib, mask=PLACES["planes"] + 1192) and planes(lib, mask=PLACES["planes"] - 1592)


OUTPUTS = ["nkept", "path", "nxt"]


@pytest.mark.parametrize("out,other", [(a, b) for a in OUTPUTS for b in ["par", "cu", "ids", "ua", "un", *OUTPUTS] if a != b])
def test_verify_over_its_vectors(lib, out, other):  # noqa: F811
    at = PLACES[other]
    assert verify(lib, **{out: at}) and verify(lib, **{out: at + VECTORS[other] - 4}) and verify(lib, **{out: at - VECTORS[out] + 4})


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("rows", ["t", "d"])
def test_verify_over_its_rows(lib, out, rows):  # noqa: F811
    base, n = FAR[rows], VECTORS[out]
    kw = dict(tst=6000, dst=6000, v=5000)  # rows of 10,000 bytes, 2,000 between them
    for row in (0, 1, 50, 99):
        for at in (row * 12000, row * 12000 + 9996, row * 12000 - n + 4):
            assert verify(lib, **{out: base + at}, **kw)



# ---------------------------------------------------------------- attention ---------------------
# (rows of out and q: 8 heads of 512 bytes a token, 256 bytes between them)
SPARSE = dict(q=1 << 40, out=1 << 41, qt=8 * 384, qh=384, ot=8 * 384, oh=384)


def attend(lib, **kw):  # noqa: F811
    st = _attend(lib, **{**{k: PLACES[k] for k in ("cu", "mask")}, "ctx": PLACES["pos"], **SPARSE, **kw})
    return st == ARG and "overlap" in lib.mrope_last_error().decode()


@pytest.mark.parametrize("name,size", [("cu", 20), ("ctx", 16), ("mask", 1600)])
def test_attend_over_its_vectors(lib, name, size):  # noqa: F811
    at = 1 << 42
    for d in (0, size - 4, 4 - 3200):
        assert attend(lib, **{name: at, "lse": at + d})
    for row in (0, 7, 8 * 99 + 3):
        for d in (0, 504, -((size - 4) // 8 * 8)):
            assert attend(lib, **{name: SPARSE["out"] + 768 * row + d})


@pytest.mark.parametrize("name", ["q", "out"])
def test_attend_lse_over_rows(lib, name):  # noqa: F811
    for row in (0, 7, 8 * 99 + 7):
        for d in (0, 508, 4 - 3200):
            assert attend(lib, lse=SPARSE[name] + 768 * row + d)
