"""The 8-bit feed-forward block on the GPU: layers as 8-bit integers, their product, the gated
projections, the activation in 8 bits, and a run of them.

Every operator is compared with the float64 oracle on the same inputs.  The tolerances
follow from the arithmetic (u = half a step of a type: fp16 2^-11, bf16 2^-8, fp32 2^-24,
relative to the value; e = 2^-24):

  product  the sum is exact.  p = (float)sum xs ws: two roundings and the products' own, 2 e
      |p|, one for the sum with the bias, e |y|, and u |y| for the type.
  gated    g and v so; act in fp32 within 6e-7 of its value (gelu of a negative g: its
      argument's rounding is worth 1e-7 g^2 more), and g's own error times |act'| <= 1.13;
      two more roundings.  Values below 1e-37 are lost.
  activation  codes and scales are those of the formula in 64 bits: equal, but where 127 u /
      max|u| lies within 1e-12 of a half (its value in 64 bits is good to 127 * 8 2^-53 <
      1e-12) and u is not exact; the scale within a rounding, 2^-24.  xhat follows bit for
      bit.
"""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
TYPES = [F16, BF16, F32]
E = 2.0 ** -24
IDS = {F16: "fp16", BF16: "bf16", F32: "fp32"}


def f64(t):
    return t.double().cpu().numpy()


def codes8(n, d, seed):
    rng = np.random.default_rng(seed)
    x = rng.integers(-128, 128, size=(n, d), dtype=np.int64)
    xs = np.exp(rng.standard_normal(n)) * 0.01
    return torch.from_numpy(x.astype(np.int8)).cuda(), torch.from_numpy(xs.astype(np.float32)).cuda()


def layer8(r, d, seed):
    """Rows whose products with codes8 are of order one."""
    rng = np.random.default_rng(seed + 7)
    w = rng.integers(-128, 128, size=(r, d), dtype=np.int64)
    ws = np.exp(0.3 * rng.standard_normal(r)) * (0.02 / np.sqrt(d))
    return torch.from_numpy(w.astype(np.int8)).cuda(), torch.from_numpy(ws.astype(np.float32)).cuda()


def product(x, xs, w, ws, bias=None):
    """(y, error of y in fp32) of the formula in float64, on the GPU: sums of integers are exact."""
    p = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    y = p if bias is None else p + bias.double()
    return f64(y), 2.02 * E * np.abs(f64(p)) + E * np.abs(f64(y))


def assert_close(y, ref, err):
    got = f64(y)
    tol = 1.001 * err + HALF[y.dtype] * np.abs(ref) * (1 + 2.0 ** -6) + 1e-36
    if y.dtype == F16:
        tol = tol + 2.0 ** -25   # subnormal results
    off = np.abs(got - ref)
    assert np.all(np.isfinite(got))
    assert np.all(off <= tol), (float((off / tol).max()), np.argwhere(off > tol)[:4].tolist())


def gated_reference(x, xs, g, gs, u, us, act, gb=None, ub=None):
    a, da = product(x, xs, g, gs, gb)
    v, dv = product(x, xs, u, us, ub)
    f = oracle.activation(a, act)
    own = 0.0 if act in ("none", "relu") else 6e-7 + (1e-7 * np.minimum(a, 0) ** 2 if act == "gelu" else 0.0)
    df = 1.13 * da + own * np.abs(f) + 1e-37
    return f * v, np.abs(v) * df + np.abs(f) * dv + df * dv + 2 * E * np.abs(f * v)


# (n, r, d): one token to several tiles of tokens, rows and columns, ragged and whole
SHAPES = [
    (1, 1, 32), (1, 33, 64), (1, 128, 4096), (1, 200, 2080), (2, 67, 1152), (3, 31, 96), (1, 4104, 288),
    (5, 129, 416), (7, 100, 512), (8, 96, 1024), (8, 257, 11008), (9, 64, 160), (13, 16, 4096), (16, 1000, 640),
    (17, 72, 256), (24, 130, 1152), (31, 255, 96), (33, 128, 2080), (64, 384, 512), (65, 129, 1056),
    (100, 1, 128), (128, 520, 320), (129, 127, 4096), (200, 300, 992), (256, 384, 1024), (257, 300, 192),
    (300, 640, 1024), (520, 260, 736), (1203, 4100, 288), (1100, 4100, 64), (1030, 513, 2048), (2, 19200, 128),
]
SHAPE_IDS = ["n{}_r{}_d{}".format(*s) for s in SHAPES]


@pytest.mark.parametrize("T", TYPES, ids=IDS.get)
@pytest.mark.parametrize("shape", SHAPES, ids=SHAPE_IDS)
def test_linear_matches_formula(shape, T):
    import post_weight_quantization_19_b200 as g
    n, r, d = shape
    (x, xs), (w, ws) = codes8(n, d, n + d), layer8(r, d, r + d)
    bias = (torch.arange(r, device="cuda") % 97 * 0.01 - 0.3).to(T) if r % 2 else None
    y = g.gptq_int8_linear(x, xs, w, ws, bias=bias, dtype=T)
    assert y.dtype == T and y.shape == (n, r)
    assert_close(y, *product(x, xs, w, ws, bias))
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=SHAPE_IDS)
def test_gated_matches_formula(shape, act):
    import post_weight_quantization_19_b200 as g
    n, r, d = shape
    T = TYPES[(n + r + len(act)) % 3]
    (x, xs), (w, ws), (u, us) = codes8(n, d, n + d), layer8(r, d, r + d), layer8(r, d, r + d + 1)
    gb = (torch.arange(r, device="cuda") % 89 * 0.01 - 0.4).to(T) if r % 2 else None
    ub = (0.3 - torch.arange(r, device="cuda") % 83 * 0.01).to(T) if r % 3 else None
    y = g.gptq_int8_gated(x, xs, w, ws, u, us, activation=act, gate_bias=gb, up_bias=ub, dtype=T)
    assert y.dtype == T and y.shape == (n, r)
    assert_close(y, *gated_reference(x, xs, w, ws, u, us, act, gb, ub))
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("n", [1, 20, 300])
def test_largest_sums_are_exact(n):
    # 65536 columns of -128 * -128 and of 127 * -128: sums of 2^30 and just below, which
    # fp32 or a wider product's rounding would not hold; ones apart they stay apart
    import post_weight_quantization_19_b200 as g
    d, r = 65536, 40
    x = torch.full((n, d), -128, dtype=I8, device="cuda")
    w = torch.full((r, d), -128, dtype=I8, device="cuda")
    w[1] = 127
    w[2, :d // 2] = 127
    w[3:, 5] = 0
    x[n - 1, 7] = 0
    w[4, 7] = 1
    one = torch.ones(max(n, r), device="cuda")
    y = g.gptq_int8_linear(x, one[:n], w, one[:r], dtype=F32)
    exact = (x.double() @ w.double().t()).float()
    assert torch.equal(y, exact)
    # (a single token is the one with a zero)
    assert float(exact[0, 0]) == 2.0 ** 30 - (2.0 ** 14 if n == 1 else 0)


@pytest.mark.parametrize("n", [1, 9, 40, 300])
def test_integers_leave_as_they_are(n):
    # unit scales, sums below 2^24 = fp32's integers: equal, not close
    import post_weight_quantization_19_b200 as g
    (x, _), (w, _) = codes8(n, 992, n), layer8(77, 992, n)
    one = torch.ones(max(n, 77), device="cuda")
    y = g.gptq_int8_linear(x, one[:n], w, one[:77], dtype=F32)
    assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("n", [1, 20, 300])
def test_scales_that_are_no_numbers_stay_in_their_token_and_row(n):
    import post_weight_quantization_19_b200 as g
    (x, xs), (w, ws) = codes8(n, 256, 3), layer8(70, 256, 4)
    clean = g.gptq_int8_linear(x, xs, w, ws, dtype=F32)
    x[n - 1] = 0                       # what a norm leaves of a row with a NaN
    xs[n - 1] = float("nan")
    ws[5], ws[69] = float("nan"), float("inf")
    y = g.gptq_int8_linear(x, xs, w, ws, dtype=F32)
    assert torch.isnan(y[n - 1]).all() and torch.isnan(y[:, 5]).all()
    keep = [i for i in range(70) if i not in (5, 69)]
    assert torch.equal(y[:n - 1][:, keep], clean[:n - 1][:, keep])
    assert not torch.isfinite(y[:, 69]).any()


def packed(r, d, bits, seed, sym=True):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 1 << bits, size=(r, d))
    z = np.full((r, 1), 1 << (bits - 1)) if sym else rng.integers(0, 1 << bits, size=(r, 1))
    s = np.exp(rng.standard_normal((r, 1))) * 0.01
    return q, z.astype(np.int32), s.astype(np.float32), oracle.pack_rows(q, bits)


@pytest.mark.parametrize("sym", [True, False])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("r,d", [(1, 32), (3, 96), (33, 64), (130, 4096), (17, 11008), (5, 65536), (9000, 160)])
def test_weights_are_codes_less_zero_points(r, d, bits, sym):
    import post_weight_quantization_19_b200 as g
    q, z, s, words = packed(r, d, bits, r + d + bits, sym)
    w, ws = g.gptq_int8_weights(*(torch.from_numpy(v).cuda() for v in (words, s, z)), d, bits)
    ref = q - z
    fits = (ref >= -128).all(1) & (ref <= 127).all(1)
    assert fits.all() or (bits == 8 and not sym)
    np.testing.assert_array_equal(w.cpu().numpy(), np.clip(ref, -128, 127))
    got = ws.cpu().numpy()
    np.testing.assert_array_equal(got[fits], s[fits, 0])
    assert np.isnan(got[~fits]).all()


def test_weights_clamp_zero_points():
    import post_weight_quantization_19_b200 as g
    q, _, s, words = packed(4, 64, 4, 1)
    z = torch.tensor([[-5], [0], [15], [99]], dtype=torch.int32, device="cuda")
    w, _ = g.gptq_int8_weights(torch.from_numpy(words).cuda(), torch.from_numpy(s).cuda(), z, 64, 4)
    np.testing.assert_array_equal(w.cpu().numpy(), q - np.array([[0], [0], [15], [15]]))


ACTS = ["none", "relu", "silu", "gelu"]


def act_inputs(n, d, seed, T, spread=1.0):
    rng = np.random.default_rng(seed)
    channel = np.exp(0.7 * rng.standard_normal(d))
    channel[:: max(1, d // 3)] *= 20
    x = rng.standard_normal((n, d)) * channel * spread
    return torch.from_numpy(x.astype(np.float32)).to(T).cuda()


def assert_codes(res, x, up, act, T):
    """codes, scales and xhat of a result against the oracle's"""
    codes, scales = oracle.activation_int8(f64(x), None if up is None else f64(up), act)
    u = oracle.activation(f64(x), act) * (1.0 if up is None else f64(up))
    top = np.abs(u).max(1, keepdims=True)
    got = res["codes"].cpu().numpy().astype(np.int64)
    diff = got != codes
    if diff.any():
        assert act in ("silu", "gelu"), np.argwhere(diff)[:4].tolist()
        q = 127.0 * u / np.where(top > 0, top, 1)
        near = np.abs(np.abs(q - np.floor(q)) - 0.5) < 1e-12
        assert np.all(near[diff]) and np.abs(got - codes).max() == 1, np.argwhere(diff & ~near)[:4].tolist()
    s = res["scales"].cpu().numpy()
    assert s.dtype == np.float32
    np.testing.assert_allclose(s, scales, rtol=1.01 * E)
    if "xhat" in res:
        want = (res["scales"][:, None] * res["codes"].float()).to(T)
        assert torch.equal(res["xhat"], want)


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,d", [(1, 32), (3, 96), (9, 512), (2, 544), (17, 1056), (5, 2048), (1, 2080), (4, 4096),
                                 (3, 11008), (301, 288), (2, 16384), (2, 16416), (3, 32800), (2, 49152), (1, 65536)])
def test_activation_matches_oracle(n, d, act, gated, T):
    import post_weight_quantization_19_b200 as g
    x = act_inputs(n, d, n + d, T)
    up = act_inputs(n, d, n + d + 1, T) if gated else None
    res = g.gptq_activation_int8(x, up, activation=act, xhat=True)
    assert res["codes"].shape == (n, d) and res["scales"].shape == (n,)
    assert_codes(res, x, up, act, T)


@pytest.mark.parametrize("act", ["none", "relu"])
def test_activation_ties_go_to_even(act):
    # multiples of half a step of 127: every second value is an exact tie
    import post_weight_quantization_19_b200 as g
    x = (torch.arange(0, 256, device="cuda").float() * 0.5).clamp(max=127).to(F16).repeat(3, 1)
    x[1] *= 0.25
    x[2] *= -4 if act == "none" else 4
    res = g.gptq_activation_int8(x, activation=act)
    want = torch.round(x[0].double()).to(I8)
    assert torch.equal(res["codes"][0], want) and torch.equal(res["codes"][1], want)
    assert torch.equal(res["codes"][2], -want if act == "none" else want)


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [96, 2048, 4096, 20000 // 32 * 32])
@pytest.mark.parametrize("act", ACTS)
def test_rows_outside_the_safe_range(act, d, T):
    # rows of zeros, of the smallest and largest numbers, of huge and tiny products
    import post_weight_quantization_19_b200 as g
    x, up = act_inputs(10, d, 5, T, 0.1), act_inputs(10, d, 6, T, 0.1)
    x[0] = 0
    up[1] = 0
    big, small = (60000.0, 6e-8) if T == F16 else (3e38, 1e-39)
    x[2], up[2] = x[2] * small * 1e4, up[2].clamp(-1, 1) * small * 100
    x[3], up[3] = x[3].clamp(-1, 1) * big, up[3].clamp(-1, 1) * big
    x[4, 1:] = 0
    x[5] = -x[5].abs()
    if T == BF16:
        x[6], up[6] = -torch.linspace(80, 110, d, device="cuda").to(T), up[6].clamp(-1, 1) * 1e38
        x[7], up[7] = -torch.linspace(5, 14, d, device="cuda").to(T), up[7].clamp(-1, 1) * 1e30
    for gate in (None, up):
        res = g.gptq_activation_int8(x, gate, activation=act, xhat=True)
        codes, scales = oracle.activation_int8(f64(x), None if gate is None else f64(gate), act)
        with np.errstate(over="ignore"):
            want = scales.astype(np.float32)
        s = res["scales"].cpu().numpy()
        ok = np.isfinite(want)
        np.testing.assert_allclose(s[ok], want[ok], rtol=2 * E, atol=1.5e-45)
        assert np.all(np.isinf(s[~ok]))
        np.testing.assert_array_equal(res["codes"].cpu().numpy(), codes)
        sums = res["scales"][:, None] * res["codes"].float()
        assert torch.equal(torch.nan_to_num(res["xhat"]), torch.nan_to_num(sums.to(T)))


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 1024, 4096, 20000 // 32 * 32])
def test_infinities_and_nan_stay_in_their_rows(d, T):
    import post_weight_quantization_19_b200 as g
    for act in ACTS:
        x, up = act_inputs(6, d, 8, T), act_inputs(6, d, 9, T)
        clean = g.gptq_activation_int8(x, up, activation=act, xhat=True)
        x[1, d - 1] = float("nan")
        up[2, 0] = float("inf")
        x[2, 0] = 1.0
        up[4, d // 2] = float("nan")
        x[5, 3], up[5, 3] = float("-inf"), 1.0
        res = g.gptq_activation_int8(x, up, activation=act, xhat=True)
        lost = [1, 2, 4] + ([5] if act != "relu" else [])   # relu of -inf is 0
        for i in lost:
            assert torch.isnan(res["scales"][i]) and not res["codes"][i].any()
            assert torch.isnan(res["xhat"][i]).all()
        for i in (0, 3):
            assert torch.equal(res["codes"][i], clean["codes"][i])
            assert torch.equal(res["scales"][i], clean["scales"][i])
        if act == "relu":
            assert torch.isfinite(res["scales"][5]) and res["codes"][5, 3] == 0


@pytest.mark.parametrize("d", [64, 2048, 4096, 32800])
def test_activation_in_another_order(d):
    import post_weight_quantization_19_b200 as g
    for T in (F16, BF16):
        x, up = act_inputs(5, d, 10, T), act_inputs(5, d, 11, T)
        perm = torch.randperm(d, generator=torch.Generator().manual_seed(d)).int().cuda()
        a = g.gptq_activation_int8(x, up, xhat=True)
        b = g.gptq_activation_int8(x, up, xhat=True, perm=perm)
        assert torch.equal(b["codes"], a["codes"][:, perm.long()])
        assert torch.equal(b["xhat"], a["xhat"][:, perm.long()])
        assert torch.equal(b["scales"], a["scales"])


def test_feed_forward_block():
    # norm to 8 bits, both projections, the activation in 8 bits, the down projection: each step
    # from the step before it
    import post_weight_quantization_19_b200 as g
    from synth import make_activations, make_weights
    n, d, f = 150, 256, 704
    X = torch.from_numpy(make_activations(n, d, seed=1)).cuda()
    gamma = torch.linspace(0.5, 1.5, d, device="cuda").half()

    def solve(r, c, seed, X16, bits):
        W = torch.from_numpy(make_weights(r, c, seed=seed)).cuda()
        H = torch.zeros((c, c), device="cuda")
        g.gptq_hessian_accumulate(X16, H)
        res = g.gptq_quantize_layer(W, H, bits=bits, group=-1, sym=bits == 8, act_order=bits == 4)
        return res, g.gptq_int8_weights(res["qweight"], res["scales"], res["zeros"], c, bits)

    normed = g.gptq_rmsnorm_int8(X, gamma, eps=1e-5, xhat=True)
    gate, up = solve(f, d, 2, normed["xhat"], 8), solve(f, d, 3, normed["xhat"], 4)
    h = g.gptq_int8_gated(normed["codes"], normed["scales"], *gate[1], *up[1], dtype=F16)
    assert_close(h, *gated_reference(normed["codes"], normed["scales"], *gate[1], *up[1], "silu"))
    q = g.gptq_activation_int8(h, activation="none", xhat=True)
    assert_codes(q, h, None, "none", F16)
    down = solve(d, f, 4, q["xhat"], 8)
    y = g.gptq_int8_linear(q["codes"], q["scales"], *down[1], dtype=F16)
    assert_close(y, *product(q["codes"], q["scales"], *down[1]))
    # the same layers from their packed words: weights rounded to fp16 there
    p = g.gptq_packed_linear(q["codes"], down[0]["qweight"], down[0]["scales"], down[0]["zeros"], 8, -1,
                             x_scales=q["scales"], dtype=F16)
    sums = np.abs(f64(q["codes"])) @ np.abs(f64(down[1][0])).T * f64(q["scales"])[:, None] * f64(down[1][1])
    assert np.all(np.abs(f64(p) - f64(y)) <= HALF[F16] * (sums + 2 * np.abs(f64(y))) * 1.01 + 1e-6)
    # and the gate and up projections of fewer bits through the packed product
    gp = g.gptq_packed_linear(normed["codes"], gate[0]["qweight"], gate[0]["scales"], gate[0]["zeros"], 8, -1,
                              x_scales=normed["scales"])
    upp = g.gptq_packed_linear(normed["codes"], up[0]["qweight"], up[0]["scales"], up[0]["zeros"], 4, -1,
                               x_scales=normed["scales"])
    assert_codes(g.gptq_activation_int8(gp, upp, activation="silu", xhat=True), gp, upp, "silu", F16)
    assert g.gptq_check_device_status() == 0
