"""Calls of the packed layer's operators that are allowed and unusual: tensors that start
at odd places, no tokens or rows, calls from several threads, offsets past 32 bits.
"""

import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8


def layer(r, d, bits, group, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G = 1 if group == -1 else d // group
    q = torch.randint(-2 ** 31, 2 ** 31, (r, d * bits // 32), generator=gen, device="cuda",
                      dtype=torch.int64).to(torch.int32)
    s = 0.01 * torch.exp(0.3 * torch.randn((r, G), generator=gen, device="cuda"))
    z = torch.randint(0, 1 << bits, (r, G), generator=gen, device="cuda").to(torch.int32)
    return q, s, z


def moved(t, by):
    """t's values `by` elements behind an aligned address."""
    room = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
    out = room[by:by + t.numel()].view(t.shape)
    return out.copy_(t)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("n", [1, 12, 40, 210])
@pytest.mark.parametrize("bits,group", [(4, 128), (3, 32), (8, -1), (2, 64)])
def test_packed_linear_where_tensors_start(n, kind, bits, group):
    # everything but x may start at any element: the same bits as from aligned addresses
    # (the paths differ in how they load and store, not in what they add)
    import post_weight_quantization_19_b200 as g
    r, d = 136, 512
    q, s, z = layer(r, d, bits, group, n)
    T = BF16 if kind == "bf16" else F16
    x = torch.randn(n, d, device="cuda").to(T)
    xs = None
    if kind == "int8":
        x, xs = torch.randint(-128, 128, (n, d), device="cuda").to(I8), torch.rand(n, device="cuda")
    perm = torch.randperm(d, device="cuda").to(torch.int32)
    for dtype in (T, F32):
        bias = torch.randn(r, device="cuda").to(dtype)
        want = g.gptq_packed_linear(x, q, s, z, bits, group, x_scales=xs, bias=bias, perm=perm, dtype=dtype)
        for by in (1, 3, 4):
            room = torch.full((n * r + 64,), 7.0, dtype=dtype, device="cuda")
            y = room[by:by + n * r].view(n, r)
            g.gptq_packed_linear(x, moved(q, by), moved(s, by), moved(z, by), bits, group,
                                 x_scales=None if xs is None else moved(xs, by), bias=moved(bias, by),
                                 perm=moved(perm, by), y=y)
            assert torch.equal(y, want)
            assert bool((room[:by] == 7).all()) and bool((room[by + n * r:] == 7).all())
    assert g.gptq_check_device_status() == 0


def test_regroup_and_norm_where_tensors_start():
    import post_weight_quantization_19_b200 as g
    for bits in (2, 3, 4, 8):
        q, _, _ = layer(37, 512, bits, 64, bits)
        g_idx = (torch.arange(512, device="cuda") // 64).to(torch.int32)[torch.randperm(512, device="cuda")]
        want, perm = g.gptq_regroup(q, g_idx, bits, 64)
        for by in (1, 3):
            out, order = moved(torch.zeros_like(q), by), moved(torch.zeros_like(g_idx), by)
            g.gptq_regroup(moved(q, by), moved(g_idx, by), bits, 64, out=out, perm=order)
            assert torch.equal(out, want) and torch.equal(order, perm)
    x, gamma = torch.randn(5, 4096, device="cuda").to(F16), torch.ones(4096, dtype=F16, device="cuda")
    perm = torch.randperm(4096, device="cuda").to(torch.int32)
    want = g.gptq_rmsnorm_int8(x, gamma, eps=1e-5, perm=perm)
    scales = moved(torch.zeros(5, device="cuda"), 3)
    got = g.gptq_rmsnorm_int8(x, gamma, eps=1e-5, perm=moved(perm, 1), outputs={"scales": scales})
    assert torch.equal(got["codes"], want["codes"]) and torch.equal(scales, want["scales"])
    with pytest.raises(g.GPTQError):      # 16-byte rows
        g.gptq_rmsnorm_int8(moved(x, 1), gamma, eps=1e-5)


def test_no_tokens_and_no_rows():
    import post_weight_quantization_19_b200 as g
    q, s, z = layer(64, 256, 4, 64, 1)
    for x, xs in ((torch.empty((0, 256), dtype=BF16, device="cuda"), None),
                  (torch.empty((0, 256), dtype=I8, device="cuda"), torch.empty(0, device="cuda"))):
        assert g.gptq_packed_linear(x, q, s, z, 4, 64, x_scales=xs).shape == (0, 64)
    x = torch.randn(3, 256, device="cuda").to(F16)
    assert g.gptq_packed_linear(x, q[:0], s[:0], z[:0], 4, 64).shape == (3, 0)
    out = g.gptq_rmsnorm_int8(x[:0], x[0].clone(), eps=1e-5, residual=x[:0], xhat=True)
    assert out["codes"].shape == (0, 256) and out["scales"].shape == (0,) and out["h"].shape == (0, 256)


def test_calls_from_several_threads():
    # each thread on its own stream, all operators: the results of one thread alone
    import post_weight_quantization_19_b200 as g
    r, d, bits, group = 200, 1024, 4, 64
    q, s, z = layer(r, d, bits, group, 3)
    gamma = torch.ones(d, dtype=F16, device="cuda")
    orders = [(torch.arange(d, device="cuda") // group).to(torch.int32)[torch.randperm(d, device="cuda")]
              for _ in range(4)]
    inputs = [torch.randn(n, d, device="cuda").to(F16) for n in (1, 12, 60, 300)]

    def once(k, stream):
        by_group, perm = g.gptq_regroup(q, orders[k], bits, group, stream=stream)
        normed = g.gptq_rmsnorm_int8(inputs[k], gamma, eps=1e-5, perm=perm, stream=stream)
        y8 = g.gptq_packed_linear(normed["codes"], by_group, s, z, bits, group, x_scales=normed["scales"],
                                  dtype=F32, stream=stream)
        y16 = g.gptq_packed_linear(inputs[k], by_group, s, z, bits, group, perm=perm, stream=stream)
        return by_group, perm, normed["codes"], normed["scales"], y8, y16

    want = [once(k, torch.cuda.current_stream()) for k in range(4)]
    torch.cuda.synchronize()
    failed = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            for _ in range(25):
                got = once(k, stream)
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want[k]))
                torch.cuda.synchronize()
        except BaseException as e:   # noqa: BLE001 -- reported below
            failed.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed, failed
    assert g.gptq_check_device_status() == 0


@pytest.mark.parametrize("n,r,d,T", [(66000, 40, 32768, F16), (66000, 40, 32768, I8), (33000, 65568, 64, BF16),
                                     (3, 131200, 65536, F16), (40, 131200, 65536, BF16)])
def test_packed_linear_past_32_bits(n, r, d, T):
    # x, y or the codes hold more than 2^31 elements or 2^32 bytes: the last tokens and
    # rows equal those of a call on them alone
    import post_weight_quantization_19_b200 as g
    bits = 8 if r * d > 2 ** 32 else 4
    q, s, z = layer(r, d, bits, -1, 5)
    xs = None
    x = torch.empty((n, d), dtype=T, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    if T is I8:
        x.random_(-128, 128, generator=gen)
        xs = torch.rand(n, generator=gen, device="cuda")
    else:
        x.normal_(generator=gen)
    y = g.gptq_packed_linear(x, q, s, z, bits, -1, x_scales=xs)
    tokens, rows = slice(max(0, n - 300), n), slice(max(0, r - 260), r)
    part = g.gptq_packed_linear(x[tokens].contiguous(), q[rows].contiguous(), s[rows].contiguous(),
                                z[rows].contiguous(), bits, -1, x_scales=None if xs is None else xs[tokens].contiguous(),
                                dtype=F32)
    assert bool(torch.isfinite(y[-1]).all())
    u = 2.0 ** -11 if y.dtype is F16 else 2.0 ** -8
    err = (y[tokens, rows].double() - part.double()).norm() / part.double().norm()
    assert float(err) <= u                         # the weight's rounding and y's, each u / sqrt(3)
    head = g.gptq_packed_linear(x[:300].contiguous(), q[rows].contiguous(), s[rows].contiguous(),
                                z[rows].contiguous(), bits, -1,
                                x_scales=None if xs is None else xs[:300].contiguous(), dtype=F32)
    err = (y[:300, rows].double() - head.double()).norm() / head.double().norm()
    assert float(err) <= u
    assert g.gptq_check_device_status() == 0


def test_rmsnorm_and_regroup_past_32_bits():
    import post_weight_quantization_19_b200 as g
    n, d = 70000, 32768
    x = torch.empty((n, d), dtype=BF16, device="cuda").normal_()
    gamma = torch.ones(d, dtype=BF16, device="cuda")
    out = g.gptq_rmsnorm_int8(x, gamma, eps=1e-5, residual=x, xhat=True)
    last = x[-50:].contiguous()
    part = g.gptq_rmsnorm_int8(last, gamma, eps=1e-5, residual=last, xhat=True)
    for k in part:
        assert torch.equal(out[k][-50:], part[k]), k
    del x, out
    r, d, bits, group = 70000, 65536, 8, 128
    q = torch.empty((r, d * bits // 32), dtype=torch.int32, device="cuda").random_()
    g_idx = (torch.arange(d, device="cuda") // group).to(torch.int32)[torch.randperm(d, device="cuda")]
    got, perm = g.gptq_regroup(q, g_idx, bits, group)
    tail = q[-3:].contiguous()
    want, order = g.gptq_regroup(tail, g_idx, bits, group)
    assert torch.equal(perm, order) and torch.equal(got[-3:], want)


# ------------------------------------------------------------------ captures in a new process

FIRST_CALLS = """
import threading, torch, post_weight_quantization_19_b200 as g
d, bits, group = 512, 4, 64
def layer(r):
    q = torch.randint(-2**31, 2**31, (r, d * bits // 32), device="cuda", dtype=torch.int64).to(torch.int32)
    return q, torch.rand(r, d // group, device="cuda"), torch.full((r, d // group), 7, device="cuda", dtype=torch.int32)
q, s, z = layer(200)
"""

REGROUP_BESIDE_A_CAPTURE = FIRST_CALLS + """
g_idx = (torch.arange(d, device="cuda") // group).to(torch.int32)[torch.randperm(d, device="cuda")]
out, perm = torch.empty_like(q), torch.empty_like(g_idx)
side, x, said = torch.cuda.Stream(), torch.zeros(8, device="cuda"), []
torch.cuda.synchronize()
def regroup():
    try:
        g.gptq_regroup(q, g_idx, bits, group, out=out, perm=perm, stream=side)
        said.append(None)
    except BaseException as e:
        said.append(repr(e))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    x += 1
    t = threading.Thread(target=regroup)
    t.start()
    t.join()
    regroup()
    x += 1
assert said == [None, None], said
graph.replay()
torch.cuda.synchronize()
assert x[0] == 2 and torch.equal(perm.long(), torch.sort(g_idx, stable=True)[1])
print("done")
"""

FIRST_CALL_IS_CAPTURED = FIRST_CALLS + """
gamma = torch.ones(d, dtype=torch.float16, device="cuda")
perm = torch.randperm(d, device="cuda").to(torch.int32)
xs = [torch.randn(n, d, device="cuda").half() for n in (3, 40, 400)]
torch.cuda.synchronize()
def calls():
    ys = []
    for x in xs:
        n = g.gptq_rmsnorm_int8(x, gamma, eps=1e-5, xhat=True)
        ys += [n["codes"], n["scales"], n["xhat"]]
        for dtype in (torch.float16, torch.float32):
            ys.append(g.gptq_packed_linear(x, q, s, z, bits, group, perm=perm, dtype=dtype))
            ys.append(g.gptq_packed_linear(n["codes"], q, s, z, bits, group, x_scales=n["scales"], dtype=dtype))
    return ys
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
print("done")
"""


@pytest.mark.parametrize("program", [REGROUP_BESIDE_A_CAPTURE, FIRST_CALL_IS_CAPTURED],
                         ids=["regroup_beside_a_capture", "first_call_is_captured"])
def test_first_calls_of_a_process_and_captures(program):
    # what a call sets up once per process neither ends a capture (of its own stream or
    # of another one) nor is refused by it
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "done", run.stderr[-2000:]
