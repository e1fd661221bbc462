"""fp32 results of the product from a packed layer, and sums over long rows.

With fp32 results a weight enters to fp32 accuracy for any number of tokens: exactly
(few tokens), or as s (q - z) rounded to fp32 once (2^-24) and split into parts of 16
bits (bf16: three, exactly; fp16: two, of which the second is at most half a step of the
first, 2^-11 of w, and is rounded to 11 bits itself: 2^-23 of w).

Sums: the tensor core adds at most 256 features of one result before they are added
in fp32, in at most PARTS * 16 instructions of 16 products each.  It truncates: what an
instruction loses is taken as at most two whole steps, 2 * 2^-23 of what is summed up
so far, and 16 steps more for what the products lose among themselves.  The d / 256 sums,
which grow evenly (so half of them counts), and up to 24 more additions (warps, CTAs,
bias, the scale of the token) are rounded, 2^-24 each.  So, with a = sum |w x|,

    |y - ref| <= 2^-24 |ref| + (3 * 2^-24 + (PARTS * 32 + 16) 2^-23 + (d / 512 + 24) 2^-24) a

and with few tokens the terms that cancel in s (sum (B + q) x - (B + z) sum x) add 24
additions of a group over sum s (2 B + q + z) |x|, B <= 64, at four half steps.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
PARTS = {F16: 2, I8: 2, BF16: 3}


def layer(r, d, bits, group, seed, exact=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G = 1 if group == -1 else d // group
    q = torch.randint(-2 ** 31, 2 ** 31, (r, d * bits // 32), generator=gen, device="cuda",
                      dtype=torch.int64).to(torch.int32)
    e = torch.randn((r, G), generator=gen, device="cuda")
    s = 2.0 ** (e.round() - 6) if exact else 0.01 * torch.exp(0.5 * e)
    z = torch.randint(0, 1 << bits, (r, G), generator=gen, device="cuda").to(torch.int32)
    return q, s, z


def codes_of(q, bits, d):
    pos = torch.arange(d, device=q.device) * bits
    word, off = pos // 32, (pos % 32)
    both = (q.long() & 0xFFFFFFFF)[:, word] | \
        (q.long() & 0xFFFFFFFF)[:, torch.clamp(word + 1, max=q.shape[1] - 1)] << 32
    return (both >> off) & ((1 << bits) - 1)


def reference(x, q, s, z, bits, group, xs=None, bias=None):
    """(y, sum |w x|, sum s (q + z + 128) |x|) in 64 bits on the device."""
    r, d = q.shape[0], x.shape[1]
    size = d if group == -1 else group
    c = codes_of(q, bits, d).double()
    step, zero = s.double().repeat_interleave(size, 1), z.double().repeat_interleave(size, 1)
    w, X = step * (c - zero), x.double()
    if xs is not None:
        X = X * xs.double()[:, None]
    y, a, parts = X @ w.t(), X.abs() @ w.abs().t(), X.abs() @ (step * (c + zero + 128)).t()
    if bias is not None:
        y, a = y + bias.double(), a + bias.double().abs()
    return y, a, parts


def activations(n, d, seed, T):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if T is I8:
        return (torch.randint(-128, 128, (n, d), generator=gen, device="cuda").to(I8),
                torch.exp(torch.randn(n, generator=gen, device="cuda")) * 0.01)
    x = torch.randn((n, d), generator=gen, device="cuda")
    x = x * torch.exp(0.7 * torch.randn(d, generator=gen, device="cuda"))
    return x.to(T), None


def few_tokens(n, T):
    return n <= (64 if T is I8 else 32)      # which kernel takes them, as the library has it


def tolerance(T, d, ref, a, parts, few):
    tol = 2.0 ** -24 * ref.abs() + (3 * 2.0 ** -24 + (PARTS[T] * 32 + 16) * 2.0 ** -23
                                    + (d / 512 + 24) * 2.0 ** -24) * a
    return tol + (4 * 24 * 2.0 ** -24 * parts if few and T is not I8 else 0)


# (n, r, d, bits, group)
SHAPES = [(9, 64, 160, 3, 160), (16, 129, 4096, 4, 128), (17, 72, 256, 4, 128), (31, 255, 96, 8, 32),
          (48, 300, 1152, 2, 64), (65, 129, 1056, 4, 96), (100, 1, 128, 4, -1), (128, 520, 320, 8, 64),
          (129, 127, 4096, 4, 128), (192, 260, 2080, 3, -1), (193, 33, 32, 4, 32), (257, 300, 192, 3, 64),
          (300, 640, 1024, 2, 128), (401, 260, 736, 4, 32), (577, 384, 160, 3, 160), (640, 136, 11008, 4, 128),
          (1203, 4100, 288, 4, 32), (1203, 500, 416, 8, 416), (2000, 1100, 512, 4, 128)]


@pytest.mark.parametrize("T", [F16, BF16, I8], ids=["fp16", "bf16", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=["n{}_r{}_d{}_b{}_g{}".format(*v) for v in SHAPES])
def test_fp32_results_hold_fp32_weights(shape, T):
    import post_weight_quantization_19_b200 as g
    n, r, d, bits, group = shape
    q, s, z = layer(r, d, bits, group, n + r)
    x, xs = activations(n, d, n + d, T)
    bias = torch.linspace(-1, 1, r, device="cuda") if r % 2 else None
    room = torch.full((n * r + 128,), 7.0, device="cuda")
    y = room[64:64 + n * r].view(n, r)
    g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, bias=bias, y=y)
    assert bool((room[:64] == 7).all()) and bool((room[-64:] == 7).all())
    ref, a, parts = reference(x, q, s, z, bits, group, xs, bias)
    err = (y.double() - ref).abs()
    assert bool((err <= tolerance(T, d, ref, a, parts, few_tokens(n, T))).all())
    if n * r >= 1000:
        # weights rounded to 16 bits would be off by 2^-11 / sqrt(3) (bf16 2^-8 / sqrt(3)) of the
        # 2-norm; the sums' steps by at most PARTS * 32 + 16 of 2^-23 each
        rel = float((y.double() - ref).norm() / ref.norm())
        assert rel <= (PARTS[T] * 32 + 16) * 2.0 ** -23, rel
    assert g.gptq_check_device_status() == 0
    again = g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, bias=bias, dtype=F32)
    assert torch.equal(again, y)


@pytest.mark.parametrize("T", [F16, BF16, I8], ids=["fp16", "bf16", "int8"])
@pytest.mark.parametrize("n,d,bits,group", [(4, 65536, 4, 128), (16, 65536, 8, -1), (40, 65536, 4, 128),
                                            (180, 49152, 3, 128), (300, 65536, 4, 64), (300, 65536, 2, -1),
                                            (260, 11008, 8, 128)])
@pytest.mark.parametrize("exact", [True, False], ids=["weights16", "weights32"])
def test_fp32_results_of_long_rows_of_one_sign(n, d, bits, group, T, exact):
    # products of one sign: what the tensor core's additions lose adds up over the row
    import post_weight_quantization_19_b200 as g
    r = 96
    q, s, _ = layer(r, d, bits, group, n + bits, exact)
    z = torch.zeros(s.shape, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(d)
    if T is I8:
        x, xs = torch.randint(20, 128, (n, d), generator=gen, device="cuda").to(I8), \
            torch.full((n,), 2.0 ** -7, device="cuda")
    else:
        x, xs = (torch.rand((n, d), generator=gen, device="cuda") + 0.5).to(T), None
    y = g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, dtype=F32)
    ref, a, parts = reference(x, q, s, z, bits, group, xs)
    err = y.double() - ref
    assert bool((err.abs() <= tolerance(T, d, ref, a, parts, few_tokens(n, T))).all())
    # the mean, signed: the rounded additions average out, and what the tensor core
    # loses is at most half of its bound, as the sum of 256 features grows evenly
    mean = float((err / ref).mean())
    assert abs(mean) <= (PARTS[T] * 32 + 16) * 2.0 ** -24, mean
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("T", [F16, BF16, I8], ids=["fp16", "bf16", "int8"])
def test_fp32_results_in_a_graph_and_in_an_order(T):
    # the same bits from two streams, from a graph on new inputs, with x in another order
    import post_weight_quantization_19_b200 as g
    n, r, d, bits, group = 330, 700, 2048, 4, 128
    q, s, z = layer(r, d, bits, group, 2)
    (xa, sa), (xb, sb) = activations(n, d, 1, T), activations(n, d, 2, T)
    perm = torch.randperm(d, device="cuda")
    kw = dict(dtype=F32, perm=perm.to(torch.int32))
    want = [g.gptq_packed_linear(x[:, perm].contiguous(), q, s, z, bits, group, x_scales=v, dtype=F32)
            for x, v in ((xa, sa), (xb, sb))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = g.gptq_packed_linear(xb, q, s, z, bits, group, x_scales=sb, stream=side, **kw)
    y1 = g.gptq_packed_linear(xa, q, s, z, bits, group, x_scales=sa, **kw)
    torch.cuda.synchronize()
    assert torch.equal(y1, want[0]) and torch.equal(y2, want[1])
    x, xs = xa.clone(), None if sa is None else sa.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, **kw)
    for src, v, w in ((xb, sb, want[1]), (xa, sa, want[0])):
        x.copy_(src)
        if xs is not None:
            xs.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w)


@pytest.mark.parametrize("n,d,bits,group", [(40, 65536, 4, 128), (300, 65536, 4, 64), (300, 49152, 3, -1),
                                            (1000, 11008, 8, 128)])
def test_16_bit_results_of_long_rows_of_one_sign(n, d, bits, group):
    # a row's sum stays in the tensor core here: the mean loss is at most 2^-24 of the
    # sum per 16 columns (weights exact in 16 bits; y's rounding averages out over the
    # results: half a step, 2^-11, over the square root of their number, five times)
    import post_weight_quantization_19_b200 as g
    r = 96
    q, s, _ = layer(r, d, bits, group, n + bits, exact=True)
    z = torch.zeros(s.shape, dtype=torch.int32, device="cuda")
    s *= 2.0 ** -7
    x = (torch.rand((n, d), generator=torch.Generator(device="cuda").manual_seed(d), device="cuda") + 0.5).to(F16)
    y = g.gptq_packed_linear(x, q, s, z, bits, group)
    ref, a, parts = reference(x, q, s, z, bits, group)
    assert bool(torch.isfinite(y).all())
    mean = float(((y.double() - ref) / ref).mean())
    assert abs(mean) <= 2.0 ** -24 * d / 16 + 5 * 2.0 ** -11 / (n * r) ** 0.5, mean


# ------------------------------------------------------------------ which kernel takes 9 to 16 tokens

@pytest.mark.parametrize("T", [F16, BF16, I8], ids=["fp16", "bf16", "int8"])
@pytest.mark.parametrize("n,r,d,bits,group", [(9, 64, 160, 3, 160), (13, 16, 4096, 4, 64), (16, 1000, 640, 3, 32),
                                              (16, 48, 2048, 8, -1), (11, 300, 1056, 2, 96),
                                              (15, 129, 4096, 4, 128), (16, 255, 288, 8, 32)])
def test_up_to_16_tokens_codes_enter_exactly(n, r, d, bits, group, T):
    # 16-bit results of 9 to 16 tokens (8-bit x, or layers of up to 2^25 codes): no weight is
    # rounded, so besides y's own rounding only the sums' is left.  The bound on those
    # is as for fp32 results of few tokens; a weight rounded to 16 bits would add up to
    # 2^-11 (bf16 2^-8) of sum |w x|.
    import post_weight_quantization_19_b200 as g
    q, s, z = layer(r, d, bits, group, n + r)
    x, xs = activations(n, d, n + d, T)
    for dtype in ((F16, BF16) if T is I8 else (T,)):
        bias = torch.linspace(-1, 1, r, device="cuda").to(dtype) if r % 2 else None
        y = g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, bias=bias, dtype=dtype)
        ref, a, parts = reference(x, q, s, z, bits, group, xs, bias)
        u = 2.0 ** -11 if dtype is F16 else 2.0 ** -8
        tol = u * ref.abs() * (1 + 2.0 ** -6) + tolerance(T, d, ref, a, parts, True)
        if dtype is F16:
            tol = tol + 2.0 ** -25                      # subnormal results
        assert bool(((y.double() - ref).abs() <= tol).all())
        # y's rounding alone: at most u of the 2-norm, and u / sqrt(3) where it is even over
        # a step; a weight's rounding of the same size, independent, would make it sqrt(2) of that
        if n * r >= 4000:
            rel = float((y.double() - ref).norm() / ref.norm())
            assert rel <= u / 3 ** 0.5, rel


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("n", [9, 16])
def test_layers_of_up_to_2_25_codes_take_the_exact_kernel(n, T):
    # On the border the tokens' results are those of the exact codes; one row tile past it,
    # those of the tensor-core product, whatever the number of tokens up to 192.
    import post_weight_quantization_19_b200 as g
    d, bits, group = 4096, 4, 128
    x, _ = activations(17, d, n, T)
    for r, exact in ((8192, True), (8224, False)):
        q, s, z = layer(r, d, bits, group, r)
        few = g.gptq_packed_linear(x[:n].contiguous(), q, s, z, bits, group)
        many = g.gptq_packed_linear(x, q, s, z, bits, group)[:n]
        assert torch.equal(few, many) != exact
        ref = reference(x[:n], q, s, z, bits, group)[0]
        rel = [float((y.double() - ref).norm() / ref.norm()) for y in (few, many)]
        u = 2.0 ** -11 if T is F16 else 2.0 ** -8
        assert rel[0] <= (u / 3 ** 0.5 if exact else u) and rel[1] <= u


# ------------------------------------------------------------------ scales of one row far apart

@pytest.mark.parametrize("T", [F16, BF16, I8], ids=["fp16", "bf16", "int8"])
@pytest.mark.parametrize("n,bits", [(4, 4), (40, 2), (40, 8), (150, 3), (300, 4), (300, 8)])
def test_groups_with_small_scales_keep_their_accuracy(n, bits, T):
    # Groups whose scale is 2^-k of the row's largest one, met by x alone (x is 0 elsewhere): their
    # weights are as good as any.  fp32 results for k = 8; 16-bit results for k = 18 with
    # 2 to 4 bits (fp16 products hold codes down to 2^(bits - 24) of the row's largest
    # scale at full precision) and k = 12 with 8.
    import post_weight_quantization_19_b200 as g
    r, d, group = 130, 512, 128
    q, s, z = layer(r, d, bits, group, n + bits)
    z = torch.full_like(z, (1 << bits) // 2)
    x, xs = activations(n, d, n, T)
    x[:, :128] = 0
    x[:, 256:384] = 0
    for dtype, k in ((F32, 8), (F16 if T is I8 else T, 12 if bits == 8 else 18)):
        scales = s.clone()
        scales[:, 1] *= 2.0 ** -k
        scales[:, 3] *= 2.0 ** -k
        scales[:, 0] = s.max()
        ref, a, parts = reference(x, q, scales, z, bits, group, xs)
        lift = 2.0 ** k if dtype is F16 else 1.0     # fp16 results in its normal range
        if dtype is F16:
            if xs is None:
                scales, ref, a, parts = scales * lift, ref * lift, a * lift, parts * lift
            else:
                xs, ref, a, parts = xs * lift, ref * lift, a * lift, parts * lift
        y = g.gptq_packed_linear(x, q, scales, z, bits, group, x_scales=xs, dtype=dtype)
        err = (y.double() - ref).abs()
        tol = tolerance(T, d, ref, a, parts, n <= 8 or (dtype is F32 and few_tokens(n, T)))
        if dtype is not F32:
            u = 2.0 ** -8 if dtype is BF16 else 2.0 ** -11
            tol = tol + u * ref.abs() * (1 + 2.0 ** -6) + (0 if n <= 8 else u * a)
            if dtype is F16:
                tol = tol + 2.0 ** -25
        assert bool((err <= tol).all()), float((err / tol).max())
