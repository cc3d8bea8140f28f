"""CPU checks of more refusals of the 8-bit cache's entry points (see test_kv8_abi_cpu for the others): host checks
only, nothing is launched."""
import pytest

from test_kv8_abi_cpu import A, ARG, OK, _apply, _attend, _decode, lib  # noqa: F401

H, T = 512, 4096  # bytes of a head (256 of bf16) and of a token of eight


@pytest.mark.parametrize("kw", [
    dict(out=A + H), dict(out=A - H), dict(out=A + 16), dict(out=A + T), dict(out=A - T), dict(out=A + 50 * T), dict(out=A - 99 * T),
    dict(out=A + 4 * H, qt=4096, ot=4096),                                   # half of the heads of one wide buffer
    dict(out=A + 8 * H - 16, qt=4096, ot=4096),
    dict(out=A + 2 * T, qt=4096, ot=2048), dict(out=A + T, qt=2048, ot=8192),  # other token strides, ranges that cross
    dict(out=A + 256, qh=512, oh=512, qt=4096, ot=4096),                     # heads half a head apart
    dict(out=A + H, qt=0, ot=0), dict(out=A + 99 * T + 7 * H),
    dict(out=A + H, n=1, ns=1), dict(out=A + 7 * H, n=1, ns=1, qt=64, ot=8),
])
def test_attend_refuses_an_output_over_its_queries(lib, kw):  # noqa: F811
    assert _attend(lib, **kw) == ARG
    assert "overlap" in lib.mrope_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(cb=0), dict(cb=256), dict(cb=8192 - 16), dict(cb=4096), dict(ct=256), dict(ch=512), dict(ct=496), dict(cb=512, ct=8192),
    dict(ch=4096, ct=256, cb=4096), dict(cb=1 << 20, ch=16 * 256 - 16, ct=256),
])
def test_appends_refuse_rows_that_overlap(lib, kw):  # noqa: F811
    for call in (_apply, _decode):
        assert call(lib, **kw) == ARG
        assert "overlap" in lib.mrope_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(), dict(ch=4096, ct=256), dict(cb=512, ct=512 * 64), dict(cb=256, ct=2 * 64 * 256, ch=64 * 256), dict(nb=1, cb=0),
    dict(nk=1, ch=0, cb=8192), dict(nk=1, ch=256, ct=256, cb=4096), dict(cb=1 << 40), dict(nb=0, cb=0),
])
def test_appends_take_any_order_of_the_dims(lib, kw):  # noqa: F811
    """(No tokens: what is checked is checked, and nothing is launched.)"""
    assert _apply(lib, n=0, **kw) == OK and _decode(lib, ns=0, **kw) == OK
