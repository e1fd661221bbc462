"""Refusals of the self-test of the 8-bit products' bounded waits, without a GPU."""

from test_int8_host import W, WS, X, XS, Y


def give_up(lib, x=X, xs=XS, n=4, w=W, ws=WS, r=8, d=128, what=1, y=Y):
    return lib.gptq_selftest_int8_timeout(x, xs, n, w, ws, r, d, what, y, None)


def test_selftest_refusals(lib):
    for bad in (dict(what=0), dict(what=-1), dict(what=4), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None),
                dict(y=None), dict(n=-1), dict(r=-1), dict(d=100), dict(d=0), dict(y=X), dict(y=WS)):
        assert give_up(lib, **bad) == 1, bad
    assert give_up(lib, n=0) == 0 and give_up(lib, r=0) == 0
