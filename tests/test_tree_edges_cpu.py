"""Refusals of the calls for trees of drafted tokens at the ends of what their kernels can address."""
import pytest

from test_tree_abi_cpu import ARG, BASE, UNSUP, _attend, lib  # noqa: F401  (lib: a fixture)

FAR = 1 << 28  # bytes from a row of a page to the next


@pytest.mark.parametrize("ct", [FAR, FAR + 16, 1 << 40])
def test_attend_rows_too_far_apart(lib, ct):  # noqa: F811
    assert _attend(lib, ct=ct, cb=64 * ct) == UNSUP
    assert "2^28" in lib.mrope_last_error().decode()


@pytest.mark.parametrize("kw", [dict(n=1 << 26, ns=4, nq=64, nk=64), dict(ns=1 << 22, nq=8, nk=8), dict(n=1 << 24, nq=64, nk=1)])
def test_attend_more_rows_than_a_grid(lib, kw):  # noqa: F811
    kw = dict(BASE, hd=64, ch=64, ct=64 * kw.get("nk", 2), cb=64 * 64 * kw.get("nk", 2), qh=64, oh=64, qt=64 * kw["nq"], ot=64 * kw["nq"],
              out=1 << 50, **kw)
    assert _attend(lib, **kw) == ARG
    assert "too many query rows" in lib.mrope_last_error().decode()
