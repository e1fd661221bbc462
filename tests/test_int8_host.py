"""The 8-bit feed-forward block without a GPU: the C entry points refuse bad arguments
before any CUDA call, the binding refuses wrong tensors, and pins of the oracle."""

import ctypes
import math

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")


def at(k, odd=0):
    """Distinct addresses far from each other, never dereferenced."""
    return ctypes.c_void_p((k << 32) + odd)


X, XS, W, WS, U, US, B, B2, Y, PERM = (at(k) for k in range(1, 11))
F16, BF16, F32, I8 = 0, 1, 2, 3


def weights(lib, q=X, s=XS, z=U, r=4, d=64, bits=8, w=W, ws=WS):
    return lib.gptq_int8_weights(q, s, z, r, d, bits, w, ws, None)


def test_weights_refusals(lib):
    for bad in (dict(r=-1), dict(r=1 << 31), dict(d=0), dict(d=40), dict(d=-32), dict(d=65568), dict(bits=5),
                dict(bits=0), dict(q=None), dict(s=None), dict(z=None), dict(w=None), dict(ws=None),
                dict(q=at(1, 2)), dict(s=at(2, 2)), dict(z=at(5, 2)), dict(w=at(3, 4)), dict(ws=at(4, 2)),
                dict(ws=W), dict(w=X), dict(w=at(1, 240)), dict(ws=at(2, 12)), dict(ws=U), dict(w=U)):
        assert weights(lib, **bad) == 1, bad
    assert weights(lib, r=0, q=None) == 0


def linear(lib, x=X, xs=XS, n=4, w=W, ws=WS, r=8, d=128, bias=None, y=Y, ytype=F16):
    return lib.gptq_int8_linear(x, xs, n, w, ws, r, d, bias, y, ytype, None)


def gated(lib, x=X, xs=XS, n=4, w=W, ws=WS, u=U, us=US, r=8, d=128, bias=None, ubias=None, act=2, y=Y,
          ytype=F16):
    return lib.gptq_int8_gated(x, xs, n, w, ws, u, us, r, d, bias, ubias, act, y, ytype, None)


@pytest.mark.parametrize("call", [linear, gated])
def test_product_refusals(lib, call):
    for bad in (dict(n=-1), dict(n=1 << 31), dict(r=-1), dict(r=1 << 31), dict(d=0), dict(d=100), dict(d=-32),
                dict(d=65568), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None),
                dict(ytype=I8), dict(ytype=-1), dict(ytype=4), dict(x=at(1, 8)), dict(xs=at(2, 2)),
                dict(w=at(3, 8)), dict(ws=at(4, 2)), dict(y=at(9, 1)), dict(y=at(9, 2), ytype=F32),
                dict(bias=at(7, 1)), dict(bias=at(7, 2), ytype=F32),
                # memory that y shares with an input: its first and its last bytes
                dict(y=X), dict(y=at(1, 510)), dict(y=at(2, 14)), dict(y=W), dict(y=at(3, 1022)),
                dict(y=WS), dict(y=B, bias=B)):
        assert call(lib, **bad) == 1, bad
    assert call(lib, n=0, x=None) == 0 and call(lib, r=0, w=None) == 0


def test_gated_refusals(lib):
    for bad in (dict(act=-1), dict(act=4), dict(u=None), dict(us=None), dict(u=at(5, 8)), dict(us=at(6, 2)),
                dict(ubias=at(8, 1)), dict(y=U), dict(y=at(6, 30)), dict(y=B2, ubias=B2)):
        assert gated(lib, **bad) == 1, bad


def act8(lib, x=X, up=U, dtype=F16, n=4, d=64, act=2, perm=None, codes=W, scales=WS, xhat=None):
    return lib.gptq_activation_int8(x, up, dtype, n, d, act, perm, codes, scales, xhat, None)


def test_activation_refusals(lib):
    for bad in (dict(dtype=F32), dict(dtype=I8), dict(dtype=-1), dict(n=-1), dict(n=1 << 31), dict(d=0),
                dict(d=40), dict(d=65568), dict(act=-1), dict(act=4), dict(x=None), dict(codes=None),
                dict(scales=None), dict(x=at(1, 8)), dict(up=at(5, 2)), dict(codes=at(3, 8)),
                dict(xhat=at(9, 8)), dict(scales=at(4, 2)), dict(perm=at(10, 2)), dict(codes=X),
                dict(codes=at(1, 496)), dict(xhat=X), dict(xhat=U), dict(xhat=W), dict(scales=W),
                dict(codes=PERM, perm=PERM)):
        assert act8(lib, **bad) == 1, bad
    assert act8(lib, n=0, x=None) == 0


def test_binding_refuses_host_tensors_and_wrong_arguments():
    import post_weight_quantization_19_b200 as g
    x, w = torch.zeros((2, 64), dtype=torch.int8), torch.zeros((4, 64), dtype=torch.int8)
    s, h = torch.zeros(4), torch.zeros((2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_int8_linear(x, s[:2], w, s)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_int8_gated(x, s[:2], w, s, w, s)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_activation_int8(h, h)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_int8_weights(torch.zeros((4, 16), dtype=torch.int32), s[:, None], s.int()[:, None], 64, 8)


def test_oracle_activation_pins():
    v = np.array([-3.0, -1.0, 0.0, 0.5, 2.0])
    np.testing.assert_array_equal(oracle.activation(v, "none"), v)
    np.testing.assert_array_equal(oracle.activation(v, "relu"), [0, 0, 0, 0.5, 2])
    # silu(v) - silu(-v) = v, silu'(0) = 1/2; gelu the same, and gelu(1) = the normal distribution's at 1
    for name in ("silu", "gelu"):
        f = oracle.activation(v, name)
        np.testing.assert_allclose(f - oracle.activation(-v, name), v, rtol=1e-15, atol=1e-16)
        e = 1e-6
        np.testing.assert_allclose((oracle.activation(np.array([e]), name) / e)[0], 0.5, rtol=1e-5)
    assert abs(oracle.activation(np.array([2.0]), "silu")[0] - 2 / (1 + math.exp(-2))) < 1e-15
    assert abs(oracle.activation(np.array([1.0]), "gelu")[0] - 0.8413447460685429) < 1e-15
    with pytest.raises(ValueError):
        oracle.activation(v, "tanh")


def test_oracle_activation_int8_pins():
    x = np.array([[1.0, -2.0, 4.0, 2.0], [0, 0, 0, 0], [-1, -2, -3, 0]])
    codes, scales = oracle.activation_int8(x, None, "none")
    np.testing.assert_array_equal(codes[0], [32, -64, 127, 64])     # 31.75, and the ties 63.5 to even
    np.testing.assert_array_equal(codes[1], 0)
    np.testing.assert_allclose(scales, [4 / 127, 1, 3 / 127], rtol=1e-15)
    codes, scales = oracle.activation_int8(x, None, "relu")
    assert not codes[2].any() and scales[2] == 1
    up = np.array([[2.0, 1, 1, 0], [1, 1, 1, 1], [1, 1, 1, 1]])
    codes, scales = oracle.activation_int8(x, up, "none")
    np.testing.assert_array_equal(codes[0], [64, -64, 127, 0])
    # half a step at most, for every activation
    rng = np.random.default_rng(3)
    x, up = rng.standard_normal((2, 6, 96)) * 3
    for name in ("none", "relu", "silu", "gelu"):
        codes, scales = oracle.activation_int8(x, up, name)
        u = oracle.activation(x, name) * up
        assert np.all(np.abs(codes * scales[:, None] - u) <= 0.5000001 * scales[:, None])
        assert np.all(np.abs(codes).max(1) == 127)


def test_oracle_int8_product_pins():
    # against integers of Python's own, and the packed layer's product
    rng = np.random.default_rng(4)
    x, w = rng.integers(-128, 128, (3, 64)), rng.integers(-128, 128, (5, 64))
    xs, ws, b = rng.random(3), rng.random(5), rng.random(5)
    y = oracle.int8_product(x, xs, w, ws, b)
    for t in range(3):
        for i in range(5):
            s = sum(int(p) * int(q) for p, q in zip(x[t], w[i]))
            assert abs(y[t, i] - (s * xs[t] * ws[i] + b[i])) < 1e-9 * (1 + abs(y[t, i]))
    packed = oracle.pack_rows(w + 128, 8)
    z = np.full((5, 1), 128)
    np.testing.assert_allclose(oracle.int8_product(x, xs, w, ws),
                               oracle.dequant_gemv(packed, ws[:, None], z, 8, -1, x * xs[:, None]), rtol=1e-12)


@pytest.mark.parametrize("name", ["int8_single.cu", "int8_pair.cu", "int8_linear.h", "int8_weights.cu",
                                  "activation_int8.cuh"])
def test_kernels_read_behind_the_wait_with_ordinary_loads(name):
    # These kernels start while the one before them on the stream still runs, so what they
    # read may be written while they live: no loads that take it for constant.
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "post_weight_quantization_19_b200", "csrc")
    with open(os.path.join(csrc, name), encoding="utf-8") as f:
        src = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert "__ldg" not in src and "__restrict__" not in src and "ld.global.nc" not in src
    for kernel in re.findall(r"__global__.*?\n}\n", src, flags=re.S):
        assert "pdl_wait_then_release()" in kernel


@pytest.mark.parametrize("name", ["int8_single.cu", "int8_pair.cu"])
def test_products_take_tensor_memory_before_the_next_kernel_may_start(name):
    # else the next kernel's CTAs could take it first, and wait for this one without end
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "post_weight_quantization_19_b200", "csrc")
    with open(os.path.join(csrc, name), encoding="utf-8") as f:
        src = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    (kernel,) = re.findall(r"__global__.*?\n}\n", src, flags=re.S)
    release = kernel.index("pdl_wait_then_release()")
    assert kernel.count("pdl_wait_then_release()") == 1
    taken = kernel.index("tmem_alloc")
    met = kernel.index("__syncthreads()" if name == "int8_single.cu" else "cluster_sync()", taken)
    assert taken < met < release
