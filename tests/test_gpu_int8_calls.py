"""Calls of the 8-bit feed-forward block's operators that are allowed and unusual: the shapes at
the borders between kernels, tensors that start at odd places, outputs' neighbours, streams,
captured graphs, threads, runs of calls without a wait between them, offsets past 32 bits.

Tolerances as in test_gpu_int8.py; what two paths must give alike is compared bit for bit
(sums of integers are exact and every later step is the same for both).
"""

import threading

import numpy as np
import pytest

from test_gpu_int8 import (ACTS, BF16, F16, F32, HALF, I8, TYPES, act_inputs, assert_close, assert_codes, codes8, f64,
                           gated_reference, layer8, product)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# (n, r, d): token counts where the number of columns per tile changes, rows per tile, a k range
# split over 2, 4 and 8 CTAs with sums beside the ring and in it, several tiles per CTA
EDGES = [
    (16, 129, 2048), (17, 4736, 1024), (32, 4800, 1024), (33, 9472, 1024), (48, 9480, 1024), (49, 300, 4096),
    (64, 2360, 4096), (5, 40000, 64), (40, 40008, 96), (60, 19000, 160), (65, 40, 11008), (100, 40, 11008),
    (128, 260, 11008), (129, 260, 11008), (250, 300, 11008), (256, 130, 16384), (300, 4104, 256), (300, 4112, 256),
    (513, 9000, 160), (1, 8, 65536), (12, 1000, 65536),
]
EDGE_IDS = ["n{}_r{}_d{}".format(*s) for s in EDGES]


@pytest.mark.parametrize("shape", EDGES, ids=EDGE_IDS)
def test_products_at_the_borders_between_kernels(shape):
    import post_weight_quantization_19_b200 as g
    n, r, d = shape
    (x, xs), (w, ws), (u, us) = codes8(n, d, n), layer8(r, d, r), layer8(r, d, r + 1)
    for T in (BF16, F32):
        bias = (torch.arange(r, device="cuda") % 61 * 0.01 - 0.2).to(T)
        assert_close(g.gptq_int8_linear(x, xs, w, ws, bias=bias, dtype=T), *product(x, xs, w, ws, bias))
        y = g.gptq_int8_gated(x, xs, w, ws, u, us, up_bias=bias, dtype=T)
        assert_close(y, *gated_reference(x, xs, w, ws, u, us, "silu", None, bias))
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("n", [1, 3, 20, 64, 65, 128, 256, 257, 400])
def test_a_token_does_not_depend_on_the_others(n):
    # the same bits for a token alone and among others, through whichever kernels
    import post_weight_quantization_19_b200 as g
    r, d = 1000, 4096
    (x, xs), (w, ws), (u, us) = codes8(400, d, 1), layer8(r, d, 2), layer8(r, d, 3)
    whole = g.gptq_int8_linear(x, xs, w, ws, dtype=F32)
    part = g.gptq_int8_linear(x[:n].contiguous(), xs[:n].contiguous(), w, ws, dtype=F32)
    assert torch.equal(part, whole[:n])
    for T in (F16, F32):
        whole = g.gptq_int8_gated(x, xs, w, ws, u, us, dtype=T)
        part = g.gptq_int8_gated(x[:n].contiguous(), xs[:n].contiguous(), w, ws, u, us, dtype=T)
        assert torch.equal(part, whole[:n])


@pytest.mark.parametrize("T", TYPES, ids=str)
@pytest.mark.parametrize("n", [1, 70, 300])
@pytest.mark.parametrize("act", ACTS)
def test_gate_values_at_the_ends_of_the_range(act, n, T):
    # infinite, NaN and huge gates of both signs, times ups of 0, -2 and infinity: as the formula
    import oracle
    import post_weight_quantization_19_b200 as g
    d, inf = 64, float("inf")
    x = torch.zeros((n, d), dtype=I8, device="cuda")
    x[:, 0] = 1
    xs = torch.ones(n, device="cuda")
    gates = [inf, -inf, float("nan"), 3.4e38, -3.4e38, 2.4e38, 1e38, -1e38, 100.0, -50.0, 0.0, 1.0]
    ups = [1.0, 0.0, -2.0, inf]
    r = len(gates) * len(ups)
    w = torch.zeros((r, d), dtype=I8, device="cuda")
    w[:, 0] = 1
    gs = torch.tensor(gates, device="cuda").repeat_interleave(len(ups))
    us = torch.tensor(ups, device="cuda").repeat(len(gates))
    y = f64(g.gptq_int8_gated(x, xs, w, gs, w, us, activation=act, dtype=T))
    with np.errstate(all="ignore"):
        want = oracle.activation(f64(gs), act) * f64(us)
        want = np.where(np.abs(want) > float(torch.finfo(T).max), np.sign(want) * np.inf, want)
    want = np.broadcast_to(want, y.shape)
    finite = np.isfinite(want)
    np.testing.assert_array_equal(y[~finite], want[~finite])
    # act to 1e-6, one product and one rounding; fp16's subnormal numbers are 2^-24 apart, so
    # the rounding of a value below 2^-14 is off by up to 2^-25 whatever its size
    tiny = 2.0 ** -25 if T == F16 else 1e-36
    assert np.all(np.abs(y[finite] - want[finite]) <= (HALF[T] + 1.2e-6) * np.abs(want[finite]) + tiny)
    assert g.gptq_check_device_status() == 0


def moved(t, by):
    """t's values `by` elements behind an aligned address."""
    room = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
    return room[by:by + t.numel()].view(t.shape).copy_(t)


@pytest.mark.parametrize("r", [136, 133, 4112])
@pytest.mark.parametrize("n", [1, 12, 40, 90, 300])
def test_products_where_tensors_start(n, r):
    # all but x and the weights may start at any element, and nothing beside y is written
    import post_weight_quantization_19_b200 as g
    d = 1024
    (x, xs), (w, ws), (u, us) = codes8(n, d, n), layer8(r, d, r), layer8(r, d, r + 1)
    for T in TYPES:
        bias = torch.randn(r, device="cuda").to(T)
        linear = g.gptq_int8_linear(x, xs, w, ws, bias=bias, dtype=T)
        both = g.gptq_int8_gated(x, xs, w, ws, u, us, gate_bias=bias, dtype=T)
        for by in (1, 4, 8):
            room = torch.full((n * r + 64,), 7.0, dtype=T, device="cuda")
            y = room[by:by + n * r].view(n, r)
            g.gptq_int8_linear(x, moved(xs, by), w, moved(ws, by), bias=moved(bias, by), y=y)
            assert torch.equal(y, linear)
            assert bool((room[:by] == 7).all()) and bool((room[by + n * r:] == 7).all())
            g.gptq_int8_gated(x, moved(xs, by), w, moved(ws, by), u, moved(us, by), gate_bias=moved(bias, by), y=y)
            assert torch.equal(y, both)
            assert bool((room[:by] == 7).all()) and bool((room[by + n * r:] == 7).all())
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("r,d", [(37, 96), (5, 4096)])
def test_weights_where_tensors_start(r, d, bits):
    import post_weight_quantization_19_b200 as g
    gen = torch.Generator(device="cuda").manual_seed(bits)
    q = torch.randint(-2 ** 31, 2 ** 31, (r, d * bits // 32), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    s = torch.rand((r, 1), generator=gen, device="cuda")
    z = torch.randint(0, 2 ** bits, (r, 1), generator=gen, device="cuda").to(torch.int32)
    want, scales = g.gptq_int8_weights(q, s, z, d, bits)
    for by in (1, 2, 4):
        room = torch.full((r * d + 128,), 99, dtype=I8, device="cuda")
        w = room[16 * by:16 * by + r * d].view(r, d)
        got = torch.full((r + 64,), 7.0, device="cuda")
        g.gptq_int8_weights(moved(q, by), moved(s, by), moved(z, by), d, bits, w=w, w_scales=got[by:by + r])
        assert torch.equal(w, want)
        assert bool((room[:16 * by] == 99).all()) and bool((room[16 * by + r * d:] == 99).all())
        assert torch.equal(torch.nan_to_num(got[by:by + r], nan=-1.0), torch.nan_to_num(scales, nan=-1.0))
        assert bool((got[:by] == 7).all()) and bool((got[by + r:] == 7).all())


def test_gate_and_up_may_be_one_layer():
    import post_weight_quantization_19_b200 as g
    for n in (2, 200):
        (x, xs), (w, ws) = codes8(n, 512, 5), layer8(300, 512, 6)
        y = g.gptq_int8_gated(x, xs, w, ws, w, ws, activation="none", dtype=F32)
        v = g.gptq_int8_linear(x, xs, w, ws, dtype=F32)
        assert torch.equal(y, v * v)


def test_no_tokens_and_no_rows():
    import post_weight_quantization_19_b200 as g
    (x, xs), (w, ws) = codes8(3, 256, 1), layer8(64, 256, 2)
    assert g.gptq_int8_linear(x[:0], xs[:0], w, ws).shape == (0, 64)
    assert g.gptq_int8_linear(x, xs, w[:0], ws[:0]).shape == (3, 0)
    assert g.gptq_int8_gated(x[:0], xs[:0], w, ws, w, ws).shape == (0, 64)
    assert g.gptq_int8_gated(x, xs, w[:0], ws[:0], w[:0], ws[:0]).shape == (3, 0)
    h = torch.empty((0, 256), dtype=F16, device="cuda")
    out = g.gptq_activation_int8(h, h, xhat=True)
    assert out["codes"].shape == (0, 256) and out["scales"].shape == (0,) and out["xhat"].shape == (0, 256)
    q = torch.empty((0, 64), dtype=torch.int32, device="cuda")
    w, s = g.gptq_int8_weights(q, torch.empty((0, 1), device="cuda"), torch.empty((0, 1), dtype=torch.int32, device="cuda"),
                               256, 8)
    assert w.shape == (0, 256) and s.shape == (0,)


def test_refusals_with_tensors():
    import post_weight_quantization_19_b200 as g
    (x, xs), (w, ws) = codes8(4, 64, 1), layer8(8, 64, 2)
    h = torch.zeros((4, 64), dtype=F16, device="cuda")
    bad = [
        lambda: g.gptq_int8_linear(x.half(), xs, w, ws), lambda: g.gptq_int8_linear(x, xs.half(), w, ws),
        lambda: g.gptq_int8_linear(x, xs[:3], w, ws), lambda: g.gptq_int8_linear(x, xs, w[:, :32], ws),
        lambda: g.gptq_int8_linear(x, xs, w.t().contiguous().t(), ws), lambda: g.gptq_int8_linear(x, xs, w, ws[:, None]),
        lambda: g.gptq_int8_linear(x, xs.cpu(), w, ws), lambda: g.gptq_int8_linear(x[0], xs, w, ws),
        lambda: g.gptq_int8_linear(x, xs, w, ws, bias=torch.zeros(8, device="cuda")),
        lambda: g.gptq_int8_linear(x, xs, w, ws, dtype=torch.float64),
        lambda: g.gptq_int8_linear(x, xs, w, ws, dtype=BF16, y=torch.zeros((4, 8), device="cuda")),
        lambda: g.gptq_int8_linear(x, xs, w, ws, y=torch.zeros((8, 4), device="cuda").t()),
        lambda: g.gptq_int8_gated(x, xs, w, ws, w[:4], ws[:4]), lambda: g.gptq_int8_gated(x, xs, w, ws, w, ws, activation="tanh"),
        lambda: g.gptq_int8_gated(x, xs, w, ws, w, ws, activation=None),
        lambda: g.gptq_activation_int8(h.float()), lambda: g.gptq_activation_int8(h, h[:2]),
        lambda: g.gptq_activation_int8(h, h.bfloat16()), lambda: g.gptq_activation_int8(h, activation="swish"),
        lambda: g.gptq_activation_int8(h[:, ::2]), lambda: g.gptq_activation_int8(h, perm=torch.arange(64, device="cuda")),
        lambda: g.gptq_int8_weights(torch.zeros((4, 16), dtype=torch.int32, device="cuda"), torch.ones((4, 2), device="cuda"),
                                    torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 64, 8),   # groups
        lambda: g.gptq_int8_weights(torch.zeros((4, 16), dtype=torch.int32, device="cuda"), torch.ones((4, 1), device="cuda"),
                                    torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 32, 8),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
    worse = [
        lambda: g.gptq_int8_linear(x[:, :48].contiguous(), xs, w[:, :48].contiguous(), ws),      # d % 32
        lambda: g.gptq_int8_linear(moved(x, 8), xs, w, ws), lambda: g.gptq_int8_linear(x, xs, moved(w, 8), ws),
        lambda: g.gptq_activation_int8(moved(h, 4)), lambda: g.gptq_activation_int8(h, outputs={"xhat": h}),
        lambda: g.gptq_int8_weights(torch.zeros((4, 10), dtype=torch.int32, device="cuda"), torch.ones((4, 1), device="cuda"),
                                    torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 64, 5),
    ]
    for call in worse:
        with pytest.raises(g.GPTQError) as e:
            call()
        assert e.value.status == 1


# ------------------------------------------------------------------ many rows of activations

@pytest.mark.parametrize("n,d", [(2700, 544), (2700, 1056), (2800, 4096), (200, 6176), (333, 11008), (160, 32800),
                                 (150, 49152), (150, 28032), (149, 65536)])
@pytest.mark.parametrize("act", ACTS)
def test_many_rows(act, n, d):
    # rows beside each other in CTAs that walk many: padding, special rows and ordinary ones
    import post_weight_quantization_19_b200 as g
    T = F16 if n % 2 else BF16
    x, up = act_inputs(n, d, 1, T), act_inputs(n, d, 2, T)
    x[::7] = 0
    x[3::50] *= 1e-3
    up[5::60] = 0
    x[9, 5], up[n - 2, d - 1] = float("nan"), float("inf")
    x[n - 2, d - 1] = 1.0
    picked = sorted({0, 1, 2, 3, 5, 7, n // 2, n // 2 + 1, n - 3, n - 1} | set(range(10, n, max(1, n // 12))))
    for gate in (None, up):
        res = g.gptq_activation_int8(x, gate, activation=act, xhat=True)
        sub = {k: v[picked] for k, v in res.items()}
        assert_codes(sub, x[picked], None if gate is None else gate[picked], act, T)
        lost = [9] if gate is None else [9, n - 2]
        assert torch.isnan(res["scales"][lost]).all() and not res["codes"][lost].any()
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[[9, n - 2]] = False
        # the same rows by themselves: the same bits, whichever kernel
        few = g.gptq_activation_int8(x[100:130].contiguous(), None if gate is None else gate[100:130].contiguous(),
                                     activation=act, xhat=True)
        for k in few:
            assert torch.equal(few[k], res[k][100:130]), k
        assert bool(torch.isfinite(res["scales"][keep]).all())
        perm = torch.randperm(d, generator=torch.Generator().manual_seed(d)).int().cuda()
        other = g.gptq_activation_int8(x, gate, activation=act, xhat=True, perm=perm)
        assert torch.equal(other["codes"], res["codes"][:, perm.long()])
        assert torch.equal(other["scales"][keep], res["scales"][keep])
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("n,d", [(7, 64), (7, 4096), (170, 11008)])
def test_activation_leaves_its_outputs_neighbours(n, d):
    import post_weight_quantization_19_b200 as g
    x, up = act_inputs(n, d, 1, F16), act_inputs(n, d, 2, F16)
    want = g.gptq_activation_int8(x, up, xhat=True)
    c, s, v = (torch.full((k,), 9, dtype=t, device="cuda") for k, t in ((n * d + 64, I8), (n + 9, F32), (n * d + 64, F16)))
    out = {"codes": c[32:32 + n * d].view(n, d), "scales": s[5:5 + n], "xhat": v[32:32 + n * d].view(n, d)}
    g.gptq_activation_int8(x, up, outputs=out)
    for k in out:
        assert torch.equal(out[k], want[k])
    for room, a, k in ((c, 32, n * d), (s, 5, n), (v, 32, n * d)):
        assert bool((room[:a] == 9).all()) and bool((room[a + k:] == 9).all())


# ------------------------------------------------------------------ streams, graphs, threads

def block(n, d, f, seed):
    """A gated block of 8-bit layers and its inputs."""
    (wg, gs), (wu, us), (wd, ds) = layer8(f, d, seed), layer8(f, d, seed + 1), layer8(d, f, seed + 2)
    ws = [wg, gs, wu, us, wd, ds]   # products of order one
    x = act_inputs(n, d, seed, F16, 0.05)
    return x, torch.linspace(0.5, 1.5, d, device="cuda").half(), ws


def forward(x, gamma, ws, out=None, stream=None):
    import post_weight_quantization_19_b200 as g
    out = out or {}
    a = g.gptq_rmsnorm_int8(x, gamma, eps=1e-5, outputs=out.get("a"), stream=stream)
    h = g.gptq_int8_gated(a["codes"], a["scales"], *ws[:4], dtype=F16, y=out.get("h"), stream=stream)
    q = g.gptq_activation_int8(h, activation="none", outputs=out.get("q"), stream=stream)
    return g.gptq_int8_linear(q["codes"], q["scales"], *ws[4:], dtype=F16, y=out.get("y"), stream=stream)


def buffers(n, d, f):
    e = lambda *s, t: torch.empty(s, dtype=t, device="cuda")   # noqa: E731
    return {"a": {"codes": e(n, d, t=I8), "scales": e(n, t=F32)}, "h": e(n, f, t=F16),
            "q": {"codes": e(n, f, t=I8), "scales": e(n, t=F32)}, "y": e(n, d, t=F16)}


@pytest.mark.parametrize("n", [1, 24, 200, 600])
def test_runs_of_calls_without_a_wait(n):
    # a block over and over in the same buffers, each run's input the last one's output: a call
    # that started before the one in front of it was done would read or overwrite what that
    # still needs.  The same steps with a wait after each give the same bits.
    d, f = 1024, 2816
    x, gamma, ws = block(n, d, f, n)
    want = x.clone()
    steps = 6
    for _ in range(steps):
        y = forward(want, gamma, ws)
        torch.cuda.synchronize()
        want = y.clone()
        torch.cuda.synchronize()
    assert bool(torch.isfinite(want).all()) and float(want.abs().max()) > 0
    for _ in range(10):
        out = buffers(n, d, f)
        cur = x.clone()
        for _ in range(steps):
            forward(cur, gamma, ws, out)
            cur.copy_(out["y"])
        assert torch.equal(cur, want)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_captured_and_replayed(n):
    d, f = 512, 1408
    x, gamma, ws = block(n, d, f, 3)
    out = buffers(n, d, f)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        forward(x, gamma, ws, out)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        forward(x, gamma, ws, out)
        forward(out["y"], gamma, ws, dict(out, y=out["h"].view(-1)[:0].new_empty((n, d))))
    for k in range(3):
        new = act_inputs(n, d, 10 + k, F16, 0.05)
        x.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["y"], forward(new, gamma, ws))


def test_two_graphs_side_by_side():
    # no memory of the library's own stands behind a call: two graphs at once do not meet
    d, f = 512, 1408
    made = []
    for k in range(2):
        x, gamma, ws = block(20, d, f, 20 + 10 * k)
        out, stream = buffers(20, d, f), torch.cuda.Stream()
        torch.cuda.synchronize()
        forward(x, gamma, ws, out, stream=stream)
        stream.synchronize()
        want = out["y"].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(10):
                forward(x, gamma, ws, out)
        made.append((graph, stream, out, want, (x, gamma, ws)))   # (the graph reads them)
    for _ in range(10):
        for graph, stream, *_ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, _ in made:
        assert torch.equal(out["y"], want)


def test_calls_from_several_threads():
    import post_weight_quantization_19_b200 as g
    d, f = 512, 1408
    blocks = [block(n, d, f, n) for n in (1, 30, 120, 400)]
    want = [forward(*b) for b in blocks]
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                y = forward(*blocks[k], stream=stream)
                stream.synchronize()
                assert torch.equal(y, want[k])
        except BaseException as e:   # noqa: BLE001 -- reported below
            failed.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed, failed
    assert g.gptq_check_device_status() == 0


def test_beside_the_other_operators():
    # between the library's own chains of kernels, in one stream without waits
    import post_weight_quantization_19_b200 as g
    from synth import make_activations, make_weights
    d, f, n = 256, 512, 300
    X = torch.from_numpy(make_activations(n, d, seed=1)).cuda()
    W = torch.from_numpy(make_weights(f, d, seed=2)).cuda()
    gamma = torch.ones(d, dtype=F16, device="cuda")

    def once(wait):
        hold = torch.cuda.synchronize if wait else (lambda: None)
        a = g.gptq_rmsnorm_int8(X, gamma, eps=1e-5, xhat=True)
        hold()
        H = torch.zeros((d, d), device="cuda")
        g.gptq_hessian_accumulate(a["xhat"], H)
        hold()
        res = g.gptq_quantize_layer(W, H, bits=8, group=-1, sym=True)
        w, ws = g.gptq_int8_weights(res["qweight"], res["scales"], res["zeros"], d, 8)
        hold()
        y = g.gptq_int8_linear(a["codes"], a["scales"], w, ws)
        hold()
        q = g.gptq_activation_int8(y, activation="relu", xhat=True)
        hold()
        H2 = torch.zeros((f, f), device="cuda")
        g.gptq_hessian_accumulate(q["xhat"], H2)
        hold()
        p = g.gptq_packed_linear(a["codes"], res["qweight"], res["scales"], res["zeros"], 8, -1, x_scales=a["scales"])
        hold()
        return w, y, q["codes"], H2, p

    want = once(True)
    for _ in range(10):
        got = once(False)
        for a, b in zip(got[:3] + got[4:], want[:3] + want[4:]):
            assert torch.equal(a, b)
        assert float((got[3] - want[3]).abs().max()) == 0


@pytest.mark.parametrize("n,r,d,T", [(66000, 40, 32768, F16), (33000, 65568, 64, BF16), (3, 131200, 65536, F16),
                                     (70, 70000, 32768, F32)])
def test_linear_past_32_bits(n, r, d, T):
    import post_weight_quantization_19_b200 as g
    gen = torch.Generator(device="cuda").manual_seed(n)

    def ints(*shape):
        return torch.randint(-128, 128, shape, generator=gen, device="cuda", dtype=I8)

    x, w = ints(n, d), ints(r, d)
    xs, ws = torch.full((n,), 0.01, device="cuda"), torch.full((r,), 0.02 / d ** 0.5, device="cuda")
    y = g.gptq_int8_linear(x, xs, w, ws, dtype=T)
    tok, row = sorted({0, 1, n // 2, n - 2, n - 1} & set(range(n))), sorted({0, 1, r // 2, r - 2, r - 1})
    assert_close(y[tok][:, row], *product(x[tok], xs[tok], w[row], ws[row]))
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("n,d", [(66000, 32768), (4300000, 512)])
def test_activation_past_32_bits(n, d):
    import post_weight_quantization_19_b200 as g
    x = torch.randn((n, d), device="cuda", dtype=BF16)
    res = g.gptq_activation_int8(x, activation="silu", xhat=True)
    rows = [0, 1, n // 2, n - 2, n - 1]
    assert_codes({k: v[rows] for k, v in res.items()}, x[rows], None, "silu", BF16)
    last = x[-64:].clone()
    few = g.gptq_activation_int8(last, activation="silu", xhat=True)
    assert all(torch.equal(few[k], res[k][-64:]) for k in few)


def test_weights_past_32_bits():
    import post_weight_quantization_19_b200 as g
    r, d = 70000, 32768
    q = torch.randint(-2 ** 31, 2 ** 31, (r, d // 8), device="cuda", dtype=torch.int64).to(torch.int32)
    s, z = torch.rand((r, 1), device="cuda"), torch.randint(0, 16, (r, 1), device="cuda").to(torch.int32)
    w, _ = g.gptq_int8_weights(q, s, z, d, 4)
    few, _ = g.gptq_int8_weights(q[-50:].clone(), s[-50:].clone(), z[-50:].clone(), d, 4)
    assert torch.equal(w[-50:], few)
    low = (q[-1].cpu().numpy().view(np.uint32)[:, None] >> (4 * np.arange(8))) & 15
    np.testing.assert_array_equal(f64(few[-1]), low.reshape(-1).astype(np.int64) - int(z[-1]))
