"""The packed layer in use on the GPU: the norm with 8-bit codes, the product
from packed weights, the columns sorted by group, and a run of them.

Every operator is compared with the float64 oracle on the same inputs.  The
tolerances follow from the arithmetic (u = half a step of a type: fp16 2^-11,
bf16 2^-8, fp32 2^-24, relative to the value):

  product, few tokens   fp32 sums of exact products: at most CHAIN(d) 2^-24
      sum |w x|, plus u |y| for the one rounding of y.  CHAIN(d) = 4 (d / 32 +
      128): a sum over d features runs through at most d / 32 + 128 additions
      one after the other in any of the kernels' orders, and the tensor core's
      fp32 additions may be off by up to four half steps (they truncate).
      With 16-bit x a group's sum is s (sum (B + q) x - (B + z) sum x), B <= 64
      (fp16: 0), so what is added up is at most s (B + q + B + z) |x| in place of |w x|:
      the part of a group (128 columns, 24 additions) adds 4 * 24 2^-24
      sum s (2 B + q + z) |x|.
  product, many tokens  the same, plus u sum |w x| for the rounding of each weight
      to 16 bits; and as those roundings are independent, a relative 2-norm error
      of at most u (about 0.8 u expected: 1/sqrt(3) for the weights, the same
      for y).
  norm   scale: a sum of squares through at most 128 additions and five more
      operations, 140 2^-24 relative.  A code may differ, by one, only where u /
      scale lies within 1e-12 of a half (its value in 64 bits is good to 127 * 8
      2^-53 < 1e-12), or within 127 * 16 * 2^-24 in rows that leave the fp32
      range.  h and xhat follow from the outputs' definition bit for bit.
"""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
EPS = 1e-5


def layer(r, d, bits, group, seed):
    rng = np.random.default_rng(seed)
    G = 1 if group == -1 else d // group
    q = rng.integers(-2 ** 31, 2 ** 31, size=(r, d * bits // 32), dtype=np.int64).astype(np.int32)
    scales = (0.01 * np.exp(0.5 * rng.standard_normal((r, G)))).astype(np.float32)
    zeros = rng.integers(0, 1 << bits, size=(r, G)).astype(np.int32)
    return q, scales, zeros


def activations(n, d, seed, T=F16):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * np.exp(0.7 * rng.standard_normal(d))
    x[:, :: max(1, d // 3)] *= 20
    return torch.from_numpy(x.astype(np.float32)).to(T).cuda()


def codes8(n, d, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.integers(-128, 128, size=(n, d), dtype=np.int64).astype(np.int8))
    xs = torch.from_numpy(np.exp(rng.standard_normal(n)).astype(np.float32) * 0.01)
    return x.cuda(), xs.cuda()


def dev(*arrays):
    return tuple(torch.from_numpy(a).cuda() for a in arrays)


def f64(t):
    return t.double().cpu().numpy()


def reference(x, q, s, z, bits, group, xs=None, bias=None, perm=None):
    """(y, sum |w x| (+ |bias|)) in float64; x a torch tensor, q/s/z numpy."""
    d = x.shape[1]
    X = f64(x)
    if xs is not None:
        X = X * f64(xs)[:, None]
    if perm is not None:
        X = X[:, perm]
    codes = oracle.unpack_rows(q, bits, d)
    gi = np.zeros(d, dtype=np.int64) if group == -1 else np.arange(d) // group
    W = s.astype(np.float64)[:, gi] * (codes - z[:, gi])
    y, a = X @ W.T, np.abs(X) @ np.abs(W).T
    if x.shape[0] <= 32 and x.dtype != I8:
        parts = np.abs(s.astype(np.float64)[:, gi]) * (2 * (64 if x.dtype == BF16 else 0) + codes + z[:, gi])
        a = a + 24 / (d / 32 + 128) * (np.abs(X) @ parts.T)
    if bias is not None:
        y, a = y + f64(bias), a + np.abs(f64(bias))
    return y, a


def assert_product(y, ref, absum, d, wtype=None):
    """wtype: the 16-bit type the weights may have been rounded to (many tokens)."""
    got, u = f64(y), HALF[y.dtype]
    assert np.all(np.isfinite(got))
    tol = u * np.abs(ref) * (1 + 2.0 ** -6) + 4 * (d / 32 + 128) * 2.0 ** -24 * absum
    if y.dtype == F16:
        tol = tol + 2.0 ** -25          # subnormal results
    if wtype is not None:
        tol = tol + HALF[wtype] * absum
        if got.size >= 1000:
            rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
            assert rel <= max(HALF[wtype], u), rel
    err = np.abs(got - ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())


def wtype_for(x):
    return F16 if x.dtype == I8 else x.dtype


# (n, r, d, bits, group)
SHAPES = [
    (1, 1, 32, 4, 32), (1, 33, 64, 4, -1), (1, 128, 4096, 4, 128), (1, 200, 2080, 3, -1),
    (2, 67, 1152, 3, 128), (3, 31, 96, 2, 96), (1, 40, 288, 8, 96), (5, 129, 416, 4, 32),
    (7, 100, 512, 2, 64), (8, 96, 1024, 8, 128), (8, 257, 11008, 4, 128), (9, 64, 160, 3, 160),
    (13, 16, 4096, 4, 64), (16, 1000, 640, 3, 32), (16, 48, 2048, 8, -1), (17, 72, 256, 4, 128),
    (24, 130, 1152, 4, 128), (31, 255, 96, 8, 32), (33, 128, 2080, 2, 32), (64, 384, 512, 3, 128),
    (65, 129, 1056, 4, 96), (100, 1, 128, 4, -1), (128, 520, 320, 8, 64), (129, 127, 4096, 4, 128),
    (257, 300, 192, 3, 64), (300, 640, 1024, 2, 128), (520, 260, 736, 4, 32),
    # tiles of two accumulators; the last tile's second one partly and wholly past the tokens
    (1203, 4100, 288, 4, 32), (1100, 4100, 64, 3, -1), (1203, 4100, 416, 8, 416),
]
IDS = ["n{}_r{}_d{}_b{}_g{}".format(*s) for s in SHAPES]


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_packed_linear_matches_oracle(shape, T):
    import post_weight_quantization_19_b200 as g
    n, r, d, bits, group = shape
    q, s, z = layer(r, d, bits, group, seed=n + r + d)
    x = activations(n, d, n + d, T)
    bias = (torch.arange(r, device="cuda") * 0.01 - 0.3).to(T) if r % 2 else None
    y = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, bias=bias)
    assert y.dtype == T and y.shape == (n, r)
    ref, absum = reference(x, q, s, z, bits, group, bias=bias)
    assert_product(y, ref, absum, d, wtype=None if n <= 8 else T)
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("n,r,d,bits,group", [
    (193, 1, 32, 4, 32), (193, 40, 4096, 3, -1), (200, 129, 96, 8, 96), (256, 257, 1056, 2, 32),
    (385, 128, 2080, 4, 416), (577, 384, 160, 3, 160), (1537, 136, 64, 4, 64)])
def test_packed_linear_beyond_one_accumulator(n, r, d, bits, group, T):
    # two row tiles at a time: one alone, an odd number of them, tokens that fill a
    # tile exactly or by one; nothing behind y is written
    import post_weight_quantization_19_b200 as g
    q, s, z = layer(r, d, bits, group, seed=n + d)
    x = activations(n, d, n + r, T)
    room = torch.full((n * r + 128,), 7.0, dtype=T, device="cuda")
    y = room[64:64 + n * r].view(n, r)
    g.gptq_packed_linear(x, *dev(q, s, z), bits, group, y=y)
    ref, absum = reference(x, q, s, z, bits, group)
    assert_product(y, ref, absum, d, wtype=T)
    assert bool((room[:64] == 7).all()) and bool((room[-64:] == 7).all())
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("T", [F16, BF16, F32], ids=["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_packed_linear_int8_matches_oracle(shape, T):
    import post_weight_quantization_19_b200 as g
    n, r, d, bits, group = shape
    q, s, z = layer(r, d, bits, group, seed=n + r + d + 1)
    x, xs = codes8(n, d, n + d)
    bias = (torch.arange(r, device="cuda") * 0.01 - 0.3).to(T) if r % 2 else None
    y = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, x_scales=xs, bias=bias, dtype=T)
    assert y.dtype == T and y.shape == (n, r)
    ref, absum = reference(x, q, s, z, bits, group, xs=xs, bias=bias)
    assert_product(y, ref, absum, d, wtype=None if n <= 8 else F16)
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("n,d,bits,group", [(1, 65536, 4, 128), (4, 65536, 8, -1), (20, 65536, 3, -1),
                                            (40, 49152, 3, 128)])
def test_packed_linear_longest_rows(n, d, bits, group):
    # one group over 65536 columns: integer sums up to 255 * 128 * 65536 < 2^31
    import post_weight_quantization_19_b200 as g
    q, s, z = layer(24, d, bits, group, seed=d + bits)
    z[:] = np.where(np.arange(24)[:, None] % 2, 0, (1 << bits) - 1)
    q[1::4], q[2::4] = -1, 0                 # codes 2^bits - 1 with zero 0, and the reverse
    x = activations(n, d, d)
    y = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, dtype=F32)
    ref, absum = reference(x, q, s, z, bits, group)
    assert_product(y, ref, absum, d, wtype=None if n <= 8 else F16)
    x8, xs = codes8(n, d, 5)
    x8[0] = -128
    y = g.gptq_packed_linear(x8, *dev(q, s, z), bits, group, x_scales=xs, dtype=F32)
    ref, absum = reference(x8, q, s, z, bits, group, xs=xs)
    assert_product(y, ref, absum, d, wtype=None if n <= 8 else F16)


@pytest.mark.parametrize("n", [1, 6, 24, 200])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
def test_packed_linear_in_a_given_order(n, kind):
    # perm: column j of the layer meets x[:, perm[j]]; entries outside [0, d) clamp
    import post_weight_quantization_19_b200 as g
    r, d, bits, group = 130, 1184, 4, 32
    q, s, z = layer(r, d, bits, group, seed=n)
    perm = np.random.default_rng(n).permutation(d).astype(np.int32)
    perm[3], perm[700] = -5, d + 7
    used = np.clip(perm, 0, d - 1)
    if kind == "int8":
        (x, xs), T = codes8(n, d, n), F16
    else:
        T = F16 if kind == "fp16" else BF16
        x, xs = activations(n, d, n, T), None
    y = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, x_scales=xs, perm=dev(perm)[0])
    ref, absum = reference(x, q, s, z, bits, group, xs=xs, perm=used)
    assert_product(y, ref, absum, d, wtype=None if n <= 8 else T)


@pytest.mark.parametrize("n", [1, 5, 40, 130])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
def test_packed_linear_keeps_tokens_and_rows_apart(n, kind):
    # A token with NaN or infinity spoils its own outputs only, a row with a NaN
    # scale its own; zero points outside the codes' range are clamped; nothing
    # before or behind y is written.
    import post_weight_quantization_19_b200 as g
    r, d, bits, group = 75, 416, 4, 32
    q, s, z = layer(r, d, bits, group, seed=3)
    z[4, :], z[9, :] = -3, 99
    bad_s = s.copy()
    bad_s[7, 2] = np.nan
    if kind == "int8":
        x, xs = codes8(n, d, n)
        T, xs2 = BF16, xs.clone()
        x2 = x.clone()
        if n > 1:
            xs2[1] = float("nan")
    else:
        T = F16 if kind == "fp16" else BF16
        x, xs, xs2 = activations(n, d, n, T), None, None
        x2 = x.clone()
        if n > 1:
            x2[1, 5], x2[n - 1, d - 1] = float("nan"), float("inf")
    zc = np.clip(z, 0, 15)
    room = torch.full((n * r + 64,), 7.0, dtype=T, device="cuda")
    y = room[32:32 + n * r].view(n, r)
    clean = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, x_scales=xs, dtype=T)
    ref, absum = reference(x, q, s, zc, bits, group, xs=xs)
    assert_product(clean, ref, absum, d, wtype=None if n <= 8 else wtype_for(x))
    g.gptq_packed_linear(x2, *dev(q, bad_s, z), bits, group, x_scales=xs2, y=y)
    assert bool((room[:32] == 7).all()) and bool((room[32 + n * r:] == 7).all())
    ok = torch.ones((n, r), dtype=torch.bool, device="cuda")
    ok[:, 7] = False
    if n > 1:
        ok[1] = False
        if kind != "int8":
            ok[n - 1] = False
        assert bool(torch.isnan(y[1]).all())
    assert bool(torch.isnan(y[:, 7]).all())
    assert torch.equal(y[ok], clean[ok])


@pytest.mark.parametrize("T,n", [(F16, 4), (BF16, 4), (F16, 70), (BF16, 70)])
def test_packed_linear_scales_of_any_size(T, n):
    # rows whose scales are far below and above the 16-bit type's own range keep
    # their relative accuracy (fp32 results)
    import post_weight_quantization_19_b200 as g
    r, d, bits, group = 96, 512, 4, 128
    q, s, z = layer(r, d, bits, group, seed=8)
    s *= (10.0 ** np.linspace(-12, 8, r)).astype(np.float32)[:, None]
    x = activations(n, d, 8, T)
    y = g.gptq_packed_linear(x, *dev(q, s, z), bits, group, dtype=F32)
    ref, absum = reference(x, q, s, z, bits, group)
    err = np.abs(f64(y) - ref)
    c = 4 * (d / 32 + 128) * 2.0 ** -24 + (0 if n <= 8 else HALF[T])
    assert np.all(err <= c * absum + 2.0 ** -24 * np.abs(ref))


@pytest.mark.parametrize("n,kind,perm", [(1, "fp16", False), (12, "bf16", True), (90, "fp16", True),
                                         (3, "int8", False), (300, "int8", True)])
def test_packed_linear_streams_graphs_and_repeats(n, kind, perm):
    # the same bits from call to call, from two streams at once, and from a
    # captured graph replayed on new inputs
    import post_weight_quantization_19_b200 as g
    r, d, bits, group = 700, 2048, 4, 128
    q, s, z = dev(*layer(r, d, bits, group, seed=2))
    order = torch.randperm(d, device="cuda").to(torch.int32) if perm else None
    T = BF16 if kind == "bf16" else F16

    def inputs(seed):
        return codes8(n, d, seed) if kind == "int8" else (activations(n, d, seed, T), None)

    def call(x, xs, **kw):
        return g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, perm=order, dtype=T, **kw)

    (xa, sa), (xb, sb) = inputs(1), inputs(2)
    ya, yb = call(xa, sa), call(xb, sb)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(one):
            y1 = call(xa, sa)
        y2 = call(xb, sb, stream=two, workspace=torch.empty(
            max(256, g.gptq_packed_linear_workspace_bytes(n, r, d, bits, group, x_dtype=xa.dtype,
                                                          permuted=perm)),
            dtype=torch.uint8, device="cuda"), y=torch.empty_like(yb))
        torch.cuda.synchronize()
        assert torch.equal(y1, ya) and torch.equal(y2, yb)
    x, xs = xa.clone(), None if sa is None else sa.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(x, xs)
    for src, scl, want in ((xb, sb, yb), (xa, sa, ya)):
        x.copy_(src)
        if xs is not None:
            xs.copy_(scl)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ------------------------------------------------------------------ the norm

def assert_norm(x, res, gamma, out, eps=EPS, perm=None, near=1e-12):
    n, d = x.shape
    T = x.dtype
    h = x if res is None else (x.float() + res.float()).to(T)
    if res is not None:
        assert torch.equal(out["h"], h)
    codes, scales = oracle.rmsnorm_int8(f64(h), f64(gamma), eps)
    got_s = f64(out["scales"])
    assert np.all(np.abs(got_s - scales) <= 140 * 2.0 ** -24 * scales)
    got = out["codes"].cpu().numpy().astype(np.int64)
    if perm is not None:
        codes = codes[:, perm]
    diff = got != codes
    if diff.any():
        u = f64(gamma) * f64(h) / np.sqrt((f64(h) ** 2).mean(1, keepdims=True) + eps)
        v = u / scales[:, None]
        if perm is not None:
            v = v[:, perm]
        assert np.abs(got - codes).max() <= 1
        off = np.abs(np.abs(v[diff]) % 1 - 0.5)
        assert off.max() <= near
    if "xhat" in out:
        assert torch.equal(out["xhat"], (out["codes"].float() * out["scales"][:, None]).to(T))


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("n,d", [(1, 32), (3, 96), (9, 256), (17, 1024), (5, 2048), (1, 2080),
                                 (4, 4096), (300, 4096), (2, 8224), (3, 11008), (1, 16384),
                                 (2, 49152), (1, 65536)])
def test_rmsnorm_int8_matches_oracle(n, d, T):
    import post_weight_quantization_19_b200 as g
    x, res = activations(n, d, d, T), activations(n, d, d + 1, T)
    gamma = (1 + 0.3 * torch.randn(d, device="cuda")).to(T)
    x[n // 2, :] *= 1e-3
    for residual in (None, res):
        out = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, residual=residual, xhat=True)
        assert_norm(x, residual, gamma, out)
        assert ("h" in out) == (residual is not None)
    perm = np.random.default_rng(d).permutation(d).astype(np.int32)
    permuted = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, residual=res, perm=dev(perm)[0], xhat=True)
    assert torch.equal(permuted["codes"], out["codes"][:, dev(perm)[0].long()])
    assert_norm(x, res, gamma, permuted, perm=perm)
    # in place: h over x, and over the residual
    for name in ("x", "residual"):
        x2, r2 = x.clone(), res.clone()
        again = g.gptq_rmsnorm_int8(x2, gamma, eps=EPS, residual=r2,
                                    outputs={"h": x2 if name == "x" else r2})
        assert torch.equal(again["h"], out["h"]) and torch.equal(again["codes"], out["codes"])
        assert torch.equal(again["scales"], out["scales"])
        assert "xhat" not in again


@pytest.mark.parametrize("d", [256, 4096])
def test_rmsnorm_int8_hard_rows(d):
    # a zero row, NaN and infinity (only their own rows are spoiled), values whose
    # squares leave the fp32 range, tiny values, a single large value, a perm
    # with entries outside [0, d)
    import post_weight_quantization_19_b200 as g
    gamma = torch.linspace(-1.5, 1.5, d, device="cuda").to(BF16)
    x = activations(8, d, 4, BF16)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, d - 1] = -float("inf")
    x[3] *= 1e30
    x[4] *= 1e-36
    x[5] = 0
    x[5, 7] = 3e38
    out = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, xhat=True)
    s, c = f64(out["scales"]), out["codes"].cpu().numpy()
    assert s[0] == 1 and not c[0].any()
    for bad in (1, 2):
        assert np.isnan(s[bad]) and not c[bad].any()
        assert bool(torch.isnan(out["xhat"][bad]).all())
    good = [0, 3, 4, 5, 6, 7]
    assert_norm(x[good], None, gamma, {k: v[good] for k, v in out.items()}, near=127 * 16 * 2.0 ** -24)
    perm = torch.arange(d, dtype=torch.int32, device="cuda")
    perm[0], perm[1] = -9, d + 5
    p = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, perm=perm)
    assert torch.equal(p["codes"], out["codes"][:, perm.long().clamp(0, d - 1)])


@pytest.mark.parametrize("d", [512, 4096])
def test_rmsnorm_int8_ties(d):
    # values in steps of 1/254 of the maximum: every second one is a tie and goes to the
    # even code, but at 0.5, 1.5 and 2.5 as the formula's last bits in 64 bits say
    # (scale = max|u| (1 / 127)); the sums of squares are exact.  Also with h over
    # x, and in another column order
    import post_weight_quantization_19_b200 as g
    rng = np.random.default_rng(d)
    x = (rng.integers(-254, 255, size=(64, d)) / 2).astype(np.float32)
    x[:, 0] = 127
    x = torch.from_numpy(x).to(F16).cuda()
    gamma = torch.full((d,), 2.0, dtype=F16, device="cuda")
    out = g.gptq_rmsnorm_int8(x, gamma, eps=EPS)
    h = f64(x)
    u = h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * 2.0
    scale = np.abs(u).max(1, keepdims=True) * (1.0 / 127)
    codes = np.where(np.abs(h) < 3, np.round(u / scale), np.round(h))
    np.testing.assert_array_equal(out["codes"].cpu().numpy(), codes)
    x2, half = x.clone() * 0.5, x.clone() * 0.5
    again = g.gptq_rmsnorm_int8(x2, gamma, eps=EPS, residual=half, xhat=True, outputs={"h": x2})
    assert torch.equal(again["codes"], out["codes"])
    assert torch.equal(again["xhat"], (out["codes"].float() * out["scales"][:, None]).to(F16))
    perm = torch.randperm(d, device="cuda").to(torch.int32)
    p = g.gptq_rmsnorm_int8(half, gamma, eps=EPS, residual=half, perm=perm)
    assert torch.equal(p["codes"], out["codes"][:, perm.long()])


def test_rmsnorm_int8_streams_and_graph():
    import post_weight_quantization_19_b200 as g
    n, d = 37, 4096
    gamma = torch.ones(d, dtype=F16, device="cuda")
    xa, xb = activations(n, d, 1), activations(n, d, 2)
    want = [g.gptq_rmsnorm_int8(v, gamma, eps=EPS, xhat=True) for v in (xa, xb)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = g.gptq_rmsnorm_int8(xb, gamma, eps=EPS, xhat=True, stream=side)
    side.synchronize()
    assert torch.equal(out["codes"], want[1]["codes"])
    x = xa.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, xhat=True)
    for src, w in ((xb, want[1]), (xa, want[0])):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("codes", "scales", "xhat"):
            assert torch.equal(out[k], w[k])


@pytest.mark.parametrize("n", [3, 40])
def test_a_calls_own_memory_belongs_to_its_stream(n, monkeypatch):
    # what a call on another stream allocates for itself is not handed out again
    # to the current stream while that stream may still use it
    import post_weight_quantization_19_b200 as g
    from post_weight_quantization_19_b200 import gptq as binding
    r, d = 96, 4096
    q, s, z = dev(*layer(r, d, 4, 128, seed=5))
    x = activations(n, d, 6)
    perm = torch.randperm(d, device="cuda").to(torch.int32)
    want = g.gptq_packed_linear(x, q, s, z, 4, 128, perm=perm)
    seen, launch = [], binding._launch
    monkeypatch.setattr(binding, "_launch",
                        lambda *args: (seen.append(args[-2:]), launch(*args))[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = g.gptq_packed_linear(x, q, s, z, 4, 128, perm=perm, stream=side)
    (pointer, size), = seen
    assert size > 0
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(abs(t.data_ptr() - pointer) >= size for t in others)
    side.synchronize()
    assert torch.equal(y, want)


# ------------------------------------------------------------------ columns by group

@pytest.mark.parametrize("r,d,bits,group", [(1, 32, 4, 32), (3, 96, 3, 32), (70, 512, 2, 64),
                                            (33, 1056, 3, 96), (257, 4096, 4, 128), (5, 65536, 8, 32),
                                            (9, 49152, 3, 128), (0, 64, 4, 32)])
def test_regroup_matches_oracle(r, d, bits, group):
    import post_weight_quantization_19_b200 as g
    rng = np.random.default_rng(r + d)
    q, _, _ = layer(r, d, bits, group, seed=d)
    g_idx = rng.permutation(np.arange(d) // group).astype(np.int32)
    room = torch.full((r * (d * bits // 32) + 16,), 5, dtype=torch.int32, device="cuda")
    out = room[8:room.numel() - 8].view(r, d * bits // 32)
    got, perm = g.gptq_regroup(*dev(q, g_idx), bits, group, out=out)
    codes, want = oracle.regroup(oracle.unpack_rows(q, bits, d), g_idx)
    np.testing.assert_array_equal(perm.cpu().numpy(), want)
    if r:
        np.testing.assert_array_equal(oracle.unpack_rows(got.cpu().numpy(), bits, d), codes)
    assert bool((room[:8] == 5).all()) and bool((room[-8:] == 5).all())


def test_regroup_refuses_unequal_groups():
    import post_weight_quantization_19_b200 as g
    q, _, _ = layer(4, 256, 4, 64, seed=1)
    for spoil in (lambda v: v.__setitem__(0, 3), lambda v: v.__setitem__(200, 99),
                  lambda v: v.__setitem__(255, -1)):
        g_idx = (np.arange(256) // 64).astype(np.int32)
        spoil(g_idx)
        with pytest.raises(g.GPTQError):
            g.gptq_regroup(*dev(q, g_idx), 4, 64)


def test_regroup_refuses_a_capture():
    import post_weight_quantization_19_b200 as g
    q, _, _ = layer(4, 256, 4, 64, seed=1)
    q, g_idx = dev(q, (np.arange(256) // 64).astype(np.int32))
    g.gptq_regroup(q, g_idx, 4, 64)
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, perm = torch.empty_like(q), torch.empty_like(g_idx)
        with pytest.raises(g.GPTQError):
            g.gptq_regroup(q, g_idx, 4, 64, out=out, perm=perm)
        x += 1
    graph.replay()
    torch.cuda.synchronize()
    assert bool((x == 1).all())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("n", [1, 20, 150])
@pytest.mark.parametrize("act", [False, True])
def test_norm_and_products_of_a_solved_layer(n, act):
    # A layer solved by the library (with and without act-order), laid out by
    # group, fed by the norm: y from the 8-bit codes and from the 16-bit values
    # equals the product with the solve's own dequantised weights.
    import post_weight_quantization_19_b200 as g
    from synth import make_activations, make_weights
    r, d, bits, group = 160, 512, 4, 64
    X = torch.from_numpy(make_activations(3000, d, seed=31)).cuda()
    W = torch.from_numpy(np.ascontiguousarray(make_weights(r, d, seed=32), dtype=np.float32)).cuda()
    H = torch.zeros((d, d), device="cuda")
    g.gptq_hessian_accumulate(X, H)
    What, g_idx = torch.empty_like(W), torch.empty(d, dtype=torch.int32, device="cuda")
    res = g.gptq_quantize_layer(W, H, bits=bits, group=group, act_order=act, W_hat=What, g_idx=g_idx)
    q, perm = g.gptq_regroup(res["qweight"], g_idx, bits, group)
    x, residual = activations(n, d, 33), activations(n, d, 34)
    gamma = (1 + 0.2 * torch.randn(d, device="cuda")).to(F16)
    normed = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, residual=residual, perm=perm, xhat=True)
    natural = g.gptq_rmsnorm_int8(x, gamma, eps=EPS, residual=residual, xhat=True)
    args = (res["scales"], res["zeros"], bits, group)
    y8 = g.gptq_packed_linear(normed["codes"], q, *args, x_scales=normed["scales"], dtype=F32)
    y8n = g.gptq_packed_linear(natural["codes"], q, *args, x_scales=natural["scales"], perm=perm,
                               dtype=F32)
    y16 = g.gptq_packed_linear(natural["xhat"], q, *args, perm=perm, dtype=F32)
    assert torch.equal(y8, y8n)
    w = f64(What)
    wq = np.abs(f64(res["scales"])).max(1, keepdims=True) * (15 + 15)   # s (q + z)
    x8 = f64(natural["codes"]) * f64(natural["scales"])[:, None]
    for y, v in ((y8, x8), (y16, f64(natural["xhat"]))):
        parts = 24 / (d / 32 + 128) * (np.abs(v) @ np.broadcast_to(wq, w.shape).T)
        assert_product(y, v @ w.T, np.abs(v) @ np.abs(w).T + parts, d, wtype=F16)


@pytest.mark.parametrize("act", [False, True])
def test_chain_with_norms_runs_on_its_codes(act):
    # Two normed layers and a plain one: each layer's inputs, codes and next inputs
    # are those its own results define, and the layer's loss is the oracle's on
    # the same inputs (the single-layer tolerance).
    import post_weight_quantization_19_b200 as g
    from parity_util import assert_codes_close
    from synth import make_activations, make_weights
    bits, group, n = 4, 64, 2500
    shapes = [(384, 256), (128, 384), (64, 128)]
    Ws = [make_weights(rr, dd, seed=41 + i) for i, (rr, dd) in enumerate(shapes)]
    gammas = [(1 + 0.2 * torch.randn(dd, device="cuda")).to(F16) for _, dd in shapes[:2]] + [None]
    X0 = torch.from_numpy(make_activations(n, 256, seed=40)).cuda()
    out = g.quantize_chain(X0, [torch.from_numpy(np.ascontiguousarray(W, dtype=np.float32)).cuda()
                                for W in Ws], bits=bits, group=group, act_order=act,
                           keep_inputs=True, norms=gammas, eps=EPS)
    X = X0
    for k, (o, W) in enumerate(zip(out, Ws)):
        d = W.shape[1]
        q = o["qweight"].cpu().numpy()
        if gammas[k] is not None:
            assert_norm(X, None, gammas[k], {"codes": o["in_codes"], "scales": o["in_scales"],
                                             "xhat": o["inputs"]})
        else:
            assert torch.equal(o["inputs"], X) and "in_codes" not in o
        if k == 0:
            ref = oracle.gptq_quantize_layer(W, oracle.hessian(o["inputs"].cpu().numpy()), bits=bits,
                                             group=group, act_order=act)
            assert_codes_close(oracle.unpack_rows(q, bits, d), ref["codes"])
            assert abs(o["loss"] - ref["loss"]) <= 5e-3 * ref["loss"]
        nxt = out[k + 1]["inputs"] if k == 1 else (None if k == 0 else o["outputs"])
        if gammas[k] is not None and nxt is not None:   # the plain layer's inputs: the product itself
            s, z = o["scales"].cpu().numpy(), o["zeros"].cpu().numpy()
            codes = oracle.unpack_rows(q, bits, d)
            gi = o["g_idx"].cpu().numpy()
            w = s.astype(np.float64)[:, gi] * (codes - z[:, gi])
            v = f64(o["in_codes"]) * f64(o["in_scales"])[:, None]
            assert_product(nxt, v @ w.T, np.abs(v) @ np.abs(w).T, d, wtype=F16)
        if k == 0:   # the next layer's norm was taken of the product
            s, z = o["scales"].cpu().numpy(), o["zeros"].cpu().numpy()
            codes = oracle.unpack_rows(q, bits, d)
            gi = o["g_idx"].cpu().numpy()
            w = s.astype(np.float64)[:, gi] * (codes - z[:, gi])
            v = f64(o["in_codes"]) * f64(o["in_scales"])[:, None]
            args = (o["qweight_by_group"] if act else o["qweight"], o["scales"], o["zeros"], bits, group)
            X = g.gptq_packed_linear(o["in_codes"], *args, x_scales=o["in_scales"], perm=o.get("perm"))
            assert_product(X, v @ w.T, np.abs(v) @ np.abs(w).T, d, wtype=F16)
        else:
            X = nxt
