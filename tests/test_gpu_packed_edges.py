"""The packed layer's operators on the GPU at values, lengths and orders where they
can go wrong, against the float64 oracle.  Half a step of a type, relative to the
value, is u: fp16 2^-11, bf16 2^-8, fp32 2^-24.
"""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
HALF = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}


def words(r, d, bits, seed):
    rng = np.random.default_rng(seed)
    return rng.integers(-2 ** 31, 2 ** 31, size=(r, d * bits // 32), dtype=np.int64).astype(np.int32)


def dev(*arrays):
    return tuple(torch.from_numpy(a).cuda() for a in arrays)


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ infinities and huge values

@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("dtype", [None, F32], ids=["same", "fp32"])
@pytest.mark.parametrize("n,bits,group", [(1, 4, 32), (1, 3, 128), (4, 2, -1), (6, 8, 64), (12, 4, 128),
                                          (16, 8, -1), (40, 4, 32), (40, 8, 128), (220, 3, -1)])
def test_packed_linear_infinite_and_huge_x(n, bits, group, T, dtype):
    # An infinity gives +-inf as the code lies above or below the zero point and
    # NaN where it is the zero point (0 inf) or where both signs meet; a finite
    # value whose products are representable gives them.  Every token of the
    # batch holds one such value in turn, so each place of a tile meets each kind.
    # Weights are exact in 16 bits (scales are powers of two), so what is left is y's own
    # rounding, 4 (d / 32 + 128) additions of at most a half step each over sum |w x|,
    # and with few tokens and bf16 the terms that cancel, s (2 B + q + z) |x| with B <= 64,
    # over a group's 24 additions.
    import post_weight_quantization_19_b200 as g
    r, d = 67, 512
    q = words(r, d, bits, n + bits)
    G = 1 if group == -1 else d // group
    s = np.full((r, G), 2.0 ** -3, dtype=np.float32)
    z = np.random.default_rng(n).integers(0, 1 << bits, size=(r, G)).astype(np.int32)
    rng = np.random.default_rng(5)
    X = np.float32(rng.standard_normal((n, d)))
    huge = np.float32(2.0 ** 14 if T == F16 else 2.0 ** (125 - bits))
    kinds = ("inf", "-inf", "both", "huge", "nan", "plain") if n > 1 else ("inf",)
    kind = [kinds[t % len(kinds)] for t in range(n)]
    for t, k in enumerate(kind):
        c = (37 * t + 5) % d
        if k == "inf":
            X[t, c] = np.inf
        elif k == "-inf":
            X[t, c] = -np.inf
        elif k == "both":
            X[t, c], X[t, (c + 200) % d] = np.inf, -np.inf
        elif k == "nan":
            X[t, c] = np.nan
        elif k == "huge" and T == BF16:
            X[t, c] = -huge
    x = torch.from_numpy(X).to(T).cuda()
    y = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, dtype=dtype)
    got = f64(y)
    codes = oracle.unpack_rows(q, bits, d)
    gi = np.zeros(d, dtype=np.int64) if group == -1 else np.arange(d) // group
    W = s.astype(np.float64)[:, gi] * (codes - z[:, gi])
    xd = f64(x)
    seen = set()
    for t, k in enumerate(kind):
        with np.errstate(invalid="ignore"):
            ref = (W * xd[t]).sum(1)
        if k in ("huge", "plain"):
            assert np.all(np.isfinite(got[t]))
            absum = np.abs(W) @ np.abs(xd[t])
            parts = (s.astype(np.float64)[:, gi] * (128 + codes + z[:, gi])) @ np.abs(xd[t])
            tol = HALF[y.dtype] * np.abs(ref) + 4 * 2.0 ** -24 * ((d / 32 + 128) * absum + 24 * parts)
            assert np.all(np.abs(got[t] - ref) <= tol), (t, k)
        else:
            np.testing.assert_array_equal(got[t], ref, err_msg=f"token {t}: {k}")
            seen.update("nan" if v != v else str(v) for v in ref)
    assert "inf" in seen and "-inf" in seen
    assert g.gptq_check_device_status() == 0


# ------------------------------------------------------------------ streams

@pytest.mark.parametrize("normed", [False, True])
def test_chain_on_a_stream_beside_a_busy_one(normed):
    # the same bits as on the current stream, while that one is kept busy
    import post_weight_quantization_19_b200 as g
    from synth import make_activations, make_weights
    shapes = [(384, 256), (128, 384)]
    Ws = [torch.from_numpy(np.ascontiguousarray(make_weights(r, d, seed=51 + i), dtype=np.float32)).cuda()
          for i, (r, d) in enumerate(shapes)]
    norms = [torch.ones(d, dtype=F16, device="cuda") for _, d in shapes] if normed else None
    X0 = torch.from_numpy(make_activations(2000, 256, seed=50)).cuda()
    kw = dict(bits=4, group=64, act_order=True, keep_inputs=True, norms=norms)
    want = g.quantize_chain(X0, Ws, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    for _ in range(200):
        busy += 1
    got = g.quantize_chain(X0, Ws, stream=side, **kw)
    side.synchronize()
    for a, b in zip(got, want):
        assert a.keys() == b.keys()
        for k in a:
            assert torch.equal(a[k], b[k]) if torch.is_tensor(a[k]) else a[k] == b[k], k
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the norm's rows outside fp32

@pytest.mark.parametrize("d", [96, 2048, 4096, 8192, 16384, 65536])
def test_rmsnorm_int8_rows_whose_products_leave_fp32(d):
    # Large values that gamma takes out (0 times them), squares beyond fp32, products
    # far below it, zero rows: scale and codes are the oracle's.  A code may differ
    # by one only where u / scale is within 1e-12 of a half (its value in 64 bits).
    # The scale is one rounding to fp32 (of a number that may be subnormal) away from
    # the value in 64 bits where the row left fp32, else 140 half steps (a sum of
    # squares through at most 128 additions and five more operations).
    import post_weight_quantization_19_b200 as g
    rng = np.random.default_rng(d)
    gamma = rng.standard_normal(d).astype(np.float32)
    gamma[0], gamma[1], gamma[2] = 0.0, 2.0 ** -130, 2.0 ** 60
    gamma = torch.from_numpy(gamma).to(BF16).cuda()
    X = rng.standard_normal((11, d)).astype(np.float32)
    X[:, 2] = 0
    X[0] *= 2.0 ** -103
    X[0, 0] = 2.0 ** 34                       # times 2^96 an infinity, and gamma is 0
    X[1] *= 2.0 ** -103
    X[1, 0] = -2.0 ** 120
    X[2], X[2, 1] = 0, 2.0 ** -120            # one product, 2^-250
    X[3] *= 2.0 ** 90                         # squares beyond fp32
    X[4, 2] = 2.0 ** 100                      # a product beyond it
    X[5] *= 2.0 ** -120
    X[6] = 0
    X[7], X[7, 0] = 0, 5.0                    # u = 0 all along
    X[8, 5] = np.inf
    X[9, 0] = np.nan                          # where gamma is 0
    x = torch.from_numpy(X).to(BF16).cuda()
    lost, outside = [8, 9], [0, 1, 2, 3, 4, 5, 6, 7]
    good = [i for i in range(11) if i not in lost]
    h, gm = f64(x), f64(gamma)
    codes, scales = oracle.rmsnorm_int8(h[good], gm, 1e-5)
    perm = np.random.default_rng(3).permutation(d).astype(np.int32)
    zero = torch.zeros_like(x)
    for kw in (dict(), dict(residual=zero), dict(residual=zero.clone(), outputs="residual"),
               dict(perm=dev(perm)[0])):
        x2 = x.clone()
        if kw.get("outputs"):
            kw["outputs"] = {"h": kw["residual"]}
        out = g.gptq_rmsnorm_int8(x2, gamma, eps=1e-5, xhat=True, **kw)
        got = out["codes"].cpu().numpy().astype(np.int64)
        if "perm" in kw:
            back = np.empty(d, dtype=np.int64)
            back[perm] = np.arange(d)
            got = got[:, back]
        s = f64(out["scales"])
        assert np.isnan(s[lost]).all() and not got[lost].any()
        assert bool(torch.isnan(out["xhat"][lost]).all())
        for k, i in enumerate(good):
            half = 2.0 ** -24 * scales[k] + 2.0 ** -150
            assert abs(s[i] - scales[k]) <= (1.0001 if i in outside else 140) * half, (i, s[i], scales[k])
            diff = got[i] != codes[k]
            if diff.any():
                u = gm * h[i] / np.sqrt((h[i] ** 2).mean() + 1e-5)
                off = np.abs(np.abs(u[diff] / scales[k]) % 1 - 0.5)
                assert np.abs(got[i] - codes[k]).max() <= 1 and off.max() <= 1e-12, i
        want = (out["codes"].float() * out["scales"][:, None]).to(BF16)
        assert torch.equal(out["xhat"].nan_to_num(7.0), want.nan_to_num(7.0))


def test_rmsnorm_int8_gamma_without_a_number():
    # a NaN or an infinity in gamma spoils every row that it meets
    import post_weight_quantization_19_b200 as g
    x = torch.ones((3, 4096), dtype=F16, device="cuda")
    for bad in (float("nan"), float("inf")):
        gamma = torch.ones(4096, dtype=F16, device="cuda")
        gamma[77] = bad
        out = g.gptq_rmsnorm_int8(x, gamma, eps=1e-5)
        assert bool(torch.isnan(out["scales"]).all()) and not bool(out["codes"].any())


# ------------------------------------------------------------------ sums of few tokens

@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("n,group", [(1, 128), (4, 32), (8, 64), (9, 128), (16, 32), (16, -1)])
def test_packed_linear_few_tokens_sums_are_fp32(n, group, bits, T):
    # Whole numbers of a unit whose partial sums all stay below 2^24 units in magnitude:
    # fp32 sums are exact in any order, with (B + q) x and (B + z) x summed apart too
    # (B <= 64), so the result is.  One value of a token is large, the others are small
    # beside it.
    import post_weight_quantization_19_b200 as g
    r, d = 70, 512
    rng = np.random.default_rng(n + bits)
    q = words(r, d, bits, bits)
    G = 1 if group == -1 else d // group
    z = rng.integers(0, 1 << bits, size=(r, G)).astype(np.int32)
    unit = 0.25 if T == F16 and bits < 8 else 1.0
    X = rng.integers(-8, 9, size=(n, d)) * unit
    X[np.arange(n), rng.integers(d, size=n)] = 32768 * rng.choice([-1, 1], size=n)
    size = d if group == -1 else group
    codes = oracle.unpack_rows(q, bits, d)
    gi = np.arange(d) // size
    assert np.abs(X).sum(1).max() * ((1 << bits) + (64 if T == BF16 else 0)) / unit < 2 ** 24
    y = g.gptq_packed_linear(torch.from_numpy(X.astype(np.float32)).to(T).cuda(),
                             *dev(q, np.ones((r, G), dtype=np.float32), z), bits, group, dtype=F32)
    np.testing.assert_array_equal(f64(y), X @ (codes - z[:, gi]).T)


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("n,d,eps", [(64, 32, 1e-5), (200, 1024, 1e-5), (300, 2080, 1e-6), (500, 4096, 1e-5),
                                     (40, 11008, 1e-5), (7, 65536, 1e-5), (64, 512, 1e20), (64, 512, 1e-30)])
def test_rmsnorm_int8_scales_are_rounded_once(n, d, eps, T):
    # The scale is the formula's value in 64 bits rounded to fp32: at most half a step
    # from it, and 2^-20 of a step for the operations in 64 bits and the correction of
    # the fp32 quotient (2^-24 of what it is off by, which is at most a few steps).
    import post_weight_quantization_19_b200 as g
    rng = np.random.default_rng(d)
    x = rng.standard_normal((n, d)) * np.exp(rng.standard_normal(d)) * 10.0 ** rng.uniform(-3, 2, size=(n, 1))
    x = torch.from_numpy(x.astype(np.float32)).to(T).cuda()
    gamma = torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)).to(T).cuda()
    out = g.gptq_rmsnorm_int8(x, gamma, eps=eps, xhat=True)
    scales = oracle.rmsnorm_int8(f64(x), f64(gamma), eps)[1]
    step = np.spacing(scales.astype(np.float32)).astype(np.float64)
    assert np.all(np.abs(f64(out["scales"]) - scales) <= step * (0.5 + 2.0 ** -20))
    want = (out["codes"].float() * out["scales"][:, None]).to(T)
    assert torch.equal(out["xhat"], want)
