"""The packed layer in use, without a GPU: the C entry points refuse bad arguments
before any CUDA call, the binding refuses wrong tensors, and pins of the
oracle's norm and column order."""

import ctypes

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(1 << 20)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
ODD2 = ctypes.c_void_p((1 << 20) + 2)
ODD1 = ctypes.c_void_p((1 << 20) + 1)
F16, BF16, F32, I8 = 0, 1, 2, 3


def norm(lib, x=P, res=P, gamma=P, dtype=F16, n=4, d=64, eps=1e-5, perm=None, h=P, codes=P,
         scales=P, xhat=None):
    return lib.gptq_rmsnorm_int8(x, res, gamma, dtype, n, d, eps, perm, h, codes, scales, xhat, None)


def test_rmsnorm_refusals(lib):
    for bad in (dict(dtype=F32), dict(dtype=I8), dict(dtype=-1), dict(n=-1), dict(n=1 << 31),
                dict(d=0), dict(d=40), dict(d=65568), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-31), dict(eps=1e31), dict(x=None), dict(gamma=None),
                dict(codes=None), dict(scales=None), dict(x=ODD), dict(res=ODD), dict(gamma=ODD),
                dict(h=ODD), dict(codes=ODD), dict(xhat=ODD), dict(scales=ODD2), dict(perm=ODD2),
                dict(xhat=P)):
        assert norm(lib, **bad) == 1, bad
    assert norm(lib, n=0, x=None) == 0


def linear(lib, x=P, xtype=F16, xs=None, n=4, q=P, s=P, z=P, perm=None, r=8, d=128, bits=4,
           group=64, bias=None, y=P, ytype=F16, ws=None, wsb=0):
    return lib.gptq_packed_linear(x, xtype, xs, n, q, s, z, perm, r, d, bits, group, bias, y, ytype,
                                  ws, wsb, None)


def test_packed_linear_refusals(lib):
    for bad in (dict(xtype=F32), dict(xtype=7), dict(ytype=BF16), dict(ytype=I8), dict(n=-1),
                dict(n=1 << 31), dict(r=-1), dict(r=1 << 31), dict(d=0), dict(d=100),
                dict(d=65568), dict(bits=5), dict(bits=0), dict(group=48), dict(group=0),
                dict(group=96), dict(group=-2), dict(x=None), dict(q=None), dict(s=None),
                dict(z=None), dict(y=None), dict(x=ODD), dict(q=ODD2), dict(s=ODD2), dict(z=ODD2),
                dict(y=ODD1), dict(bias=ODD1), dict(perm=ODD2), dict(xs=P),
                dict(xtype=I8), dict(xtype=I8, xs=ODD2), dict(xtype=I8, xs=P, ytype=I8),
                dict(ytype=F32, y=ODD2), dict(ws=ODD)):
        assert linear(lib, **bad) == 1, bad
    assert linear(lib, n=0, x=None) == 0 and linear(lib, r=0, q=None) == 0
    query = lib.gptq_packed_linear_workspace_bytes
    for bad in ((4, 8, 100, 4, -1, F16, 0), (4, 8, 128, 5, -1, F16, 0), (4, 8, 128, 4, 48, F16, 0),
                (-1, 8, 128, 4, -1, F16, 0), (4, 8, 128, 4, -1, F32, 1)):
        assert query(*bad) == 0, bad
    for args in ((4, 8, 128, 4, 64, F16, 1), (3000, 8, 128, 4, 64, I8, 0)):
        need = query(*args)
        if need:
            n, r, d, bits, group, xtype, permuted = args
            kw = dict(n=n, r=r, d=d, bits=bits, group=group, xtype=xtype,
                      xs=P if xtype == I8 else None, perm=P if permuted else None)
            assert linear(lib, ws=P, wsb=need - 1, **kw) == 4
            assert linear(lib, ws=None, wsb=0, **kw) == 4


def test_regroup_refusals(lib):
    def call(q=P, gi=P, r=4, d=128, bits=4, group=64, out=P, perm=P):
        return lib.gptq_regroup(q, gi, r, d, bits, group, out, perm, None)
    for bad in (dict(r=-1), dict(d=100), dict(d=65568), dict(bits=5), dict(group=-1),
                dict(group=48), dict(group=96), dict(q=None), dict(gi=None), dict(out=None),
                dict(perm=None), dict(q=ODD2), dict(gi=ODD2), dict(out=ODD2), dict(perm=ODD2)):
        assert call(**bad) == 1, bad


def test_binding_refuses_host_tensors_and_wrong_types():
    import post_weight_quantization_19_b200 as g
    x, w = torch.zeros((2, 64), dtype=torch.float16), torch.zeros((4, 8), dtype=torch.int32)
    s = torch.zeros((4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_packed_linear(x, w, s, s.int(), 4, -1)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_rmsnorm_int8(x, x[0], eps=1e-5)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_regroup(w, torch.zeros(64, dtype=torch.int32), 4, 64)
    with pytest.raises(ValueError):
        g.gptq_packed_linear_workspace_bytes(2, 4, 64, 4, -1, x_dtype=torch.float32)


def test_oracle_norm_pins():
    # constant rows: u = gamma exactly (eps 0 limit), scale = max|gamma| / 127; the
    # codes do not depend on the row's size; a zero row has scale 1
    gamma = np.array([1.0, -0.5, 0.25, 127 / 128])
    h = np.array([[3.0, 3, 3, 3], [0, 0, 0, 0], [1e-3, 1e-3, 1e-3, 1e-3]])
    codes, scales = oracle.rmsnorm_int8(h, gamma, 1e-300)
    np.testing.assert_allclose(scales[[0, 2]], 1 / 127, rtol=1e-12)
    assert scales[1] == 1 and not codes[1].any()
    np.testing.assert_array_equal(codes[0], [127, -64, 32, 126])
    np.testing.assert_array_equal(codes[2], codes[0])
    # the values differ from u by at most half a step
    rng = np.random.default_rng(0)
    h = rng.standard_normal((5, 64))
    codes, scales = oracle.rmsnorm_int8(h, np.ones(64), 1e-5)
    u = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5)
    assert np.all(np.abs(codes * scales[:, None] - u) <= scales[:, None] * 0.5000001)
    assert np.all(np.abs(codes).max(1) == 127)


def test_oracle_regroup_pins():
    # groups become contiguous, the order inside one is kept, and the layer's
    # product is unchanged when x follows the same order
    rng = np.random.default_rng(1)
    r, d, group, bits = 3, 96, 32, 4
    g_idx = rng.permutation(np.arange(d) // group)
    codes = rng.integers(0, 16, (r, d))
    out, perm = oracle.regroup(codes, g_idx)
    np.testing.assert_array_equal(g_idx[perm], np.arange(d) // group)
    for k in range(d // group):
        assert np.all(np.diff(perm[k * group:(k + 1) * group]) > 0)
    s, z = rng.random((r, 3)), rng.integers(0, 16, (r, 3))
    x = rng.standard_normal((2, d))
    a = oracle.dequant_gemv(oracle.pack_rows(codes, bits), s, z, bits, group, x, g_idx=g_idx)
    b = oracle.dequant_gemv(oracle.pack_rows(out, bits), s, z, bits, group, x[:, perm])
    np.testing.assert_allclose(a, b, rtol=1e-12)
