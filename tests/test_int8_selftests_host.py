"""Refusals of the self-tests of the 8-bit block, without a GPU."""

from test_int8_host import W, WS, X, XS, Y, at


def give_up(lib, x=X, xs=XS, n=4, w=W, ws=WS, r=8, d=128, what=1, y=Y):
    return lib.gptq_selftest_int8_timeout(x, xs, n, w, ws, r, d, what, y, None)


def test_selftest_refusals(lib):
    for bad in (dict(what=0), dict(what=-1), dict(what=4), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None),
                dict(y=None), dict(n=-1), dict(r=-1), dict(d=100), dict(d=0), dict(y=X), dict(y=WS)):
        assert give_up(lib, **bad) == 1, bad
    assert give_up(lib, n=0) == 0 and give_up(lib, r=0) == 0


def test_selftest_of_activations_refusals(lib):
    def call(v=X, n=4, act=2, values=Y, values64=W):
        return lib.gptq_selftest_activation(v, n, act, values, values64, None)
    for bad in (dict(n=-1), dict(n=1 << 31), dict(act=-1), dict(act=4), dict(v=None), dict(values=None),
                dict(values64=None), dict(v=at(1, 2)), dict(values=at(9, 2)), dict(values64=at(3, 4)),
                dict(values=X), dict(values64=X), dict(values64=Y), dict(values64=at(9, 40))):
        assert call(**bad) == 1, bad
    assert call(n=0, v=None) == 0
