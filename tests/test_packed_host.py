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


@pytest.mark.parametrize("act,static,group", [(False, False, 32), (True, False, 32), (True, True, 32),
                                              (True, False, -1)])
def test_chain_driver_with_norms(monkeypatch, act, static, group):
    # A normed layer: norm to 8 bits, H from the codes' values, solve, columns by
    # group under act-order, product from the codes -- with the entry points played
    # by the oracle, equal to the steps written out.
    from post_weight_quantization_19_b200 import chain
    from synth import make_activations, make_weights
    bits, eps = 4, 1e-5
    exact, calls = {}, []

    def hessian(X, H, stream=None):
        exact[H.data_ptr()] = oracle.hessian(X.numpy())

    def quantize_layer(W, H, *, bits, group, block, damp, act_order, sym, static_groups, g_idx,
                       stream=None):
        o = oracle.gptq_quantize_layer(W.numpy(), exact.pop(H.data_ptr()), bits=bits, group=group,
                                       block=block, damp=damp, act_order=act_order, sym=sym,
                                       static_groups=static_groups)
        g_idx.copy_(torch.from_numpy(o["g_idx"]))
        return {"qweight": torch.from_numpy(oracle.pack_rows(o["codes"], bits)),
                "scales": torch.from_numpy(o["scales"]), "zeros": torch.from_numpy(o["zeros"]),
                "loss": o["loss"], "g_idx": g_idx}

    def rmsnorm(x, gamma, *, eps, xhat, stream=None):
        c, s = oracle.rmsnorm_int8(x.numpy(), gamma.numpy(), eps)
        s = s.astype(np.float32)
        return {"codes": torch.from_numpy(c.astype(np.int8)), "scales": torch.from_numpy(s),
                "xhat": torch.from_numpy((c * s[:, None]).astype(np.float16))}

    def regroup(qweight, g_idx, bits, group, stream=None):
        calls.append("regroup")
        d = g_idx.numel()
        c, perm = oracle.regroup(oracle.unpack_rows(qweight.numpy(), bits, d), g_idx.numpy())
        return torch.from_numpy(oracle.pack_rows(c, bits)), torch.from_numpy(perm.astype(np.int32))

    def product(x, qweight, scales, zeros, bits, group, *, x_scales, perm, stream=None):
        v = x.numpy().astype(np.float64) * x_scales.numpy()[:, None]
        if perm is not None:
            v = v[:, perm.numpy()]
        y = oracle.dequant_gemv(qweight.numpy(), scales.numpy(), zeros.numpy(), bits, group, v)
        return torch.from_numpy(y.astype(np.float16))

    for name, f in (("gptq_hessian_accumulate", hessian), ("gptq_quantize_layer", quantize_layer),
                    ("gptq_rmsnorm_int8", rmsnorm), ("gptq_regroup", regroup),
                    ("gptq_packed_linear", product)):
        monkeypatch.setattr(chain, name, f)
    X = make_activations(500, 64, seed=5)
    Ws = [make_weights(96, 64, seed=6), make_weights(32, 96, seed=7)]
    gammas = [np.linspace(0.5, 1.5, 64).astype(np.float16), np.ones(96, dtype=np.float16)]
    got = chain.quantize_chain(torch.from_numpy(X), [torch.from_numpy(W) for W in Ws], bits=bits,
                               group=group, act_order=act, static_groups=static, keep_inputs=True,
                               norms=[torch.from_numpy(v) for v in gammas], eps=eps)
    for k, (W, gamma) in enumerate(zip(Ws, gammas)):
        c, s = oracle.rmsnorm_int8(X, gamma, eps)
        s = s.astype(np.float32)
        xhat = (c * s[:, None]).astype(np.float16)
        np.testing.assert_array_equal(got[k]["inputs"].numpy(), xhat)
        np.testing.assert_array_equal(got[k]["in_codes"].numpy(), c)
        o = oracle.gptq_quantize_layer(W, oracle.hessian(xhat), bits=bits, group=group, act_order=act,
                                       static_groups=static)
        np.testing.assert_array_equal(got[k]["qweight"].numpy(), oracle.pack_rows(o["codes"], bits))
        y = (c * s[:, None].astype(np.float64)) @ o["What"].T
        X = y.astype(np.float16)
        assert ("perm" in got[k]) == (act and group != -1 and not static)
    np.testing.assert_allclose(got[-1]["outputs"].numpy().astype(np.float64), X.astype(np.float64),
                               rtol=2.0 ** -10, atol=1e-6)
    assert len(calls) == (2 if act and group != -1 and not static else 0)


def test_chain_driver_refuses_other_counts_of_norms():
    from post_weight_quantization_19_b200 import chain
    with pytest.raises(ValueError):
        chain.quantize_chain(torch.zeros((8, 64), dtype=torch.float16), [torch.zeros((32, 64))],
                             bits=4, group=32, norms=[])
