"""CPU checks of more refusals of the 8-bit cache's entry points (see test_kv8_abi_cpu for the others): host checks
only, nothing is launched."""
import pytest

from test_kv8_abi_cpu import A, ARG, _attend, lib  # noqa: F401

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
