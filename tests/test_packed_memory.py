"""Where the packed layer's operators and the chain take and touch memory, without a
GPU: streams of a call's own tensors, memory that two arguments share, loads of what
another kernel is still writing.
"""

import contextlib
import ctypes
import os
import re

import pytest


torch = pytest.importorskip("torch")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "post_weight_quantization_19_b200", "csrc")


def code_of(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("normed", [False, True])
def test_chain_makes_its_tensors_on_its_stream(monkeypatch, normed):
    # Everything that a chain on a given stream allocates, fills and launches is under
    # that stream: a fill on the current one may come before or after its use.
    from post_weight_quantization_19_b200 import chain
    given, current, outside = object(), [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def watch(name, result):
        def call(*args, stream=None, **kw):
            if current[-1] is not given or stream is not given:
                outside.append(name)
            return result(*args, **kw)
        return call

    def made(name, make):
        def call(*args, **kw):
            if current[-1] is not given:
                outside.append(name)
            return make(*args, **kw)
        return call

    def solve(W, H, *, bits, group, g_idx, **kw):
        r, d = W.shape
        g_idx.copy_(torch.arange(d) // group)
        return {"qweight": torch.zeros((r, d * bits // 32), dtype=torch.int32), "g_idx": g_idx,
                "scales": torch.ones((r, d // group)), "zeros": torch.zeros((r, d // group)).int()}

    fakes = {"gptq_hessian_accumulate": lambda X, H: None, "gptq_quantize_layer": solve,
             "gptq_dequant_fp16": lambda q, s, z, d, *a, **kw: torch.zeros((q.shape[0], d)).half(),
             "gptq_linear_fp16": lambda X, W: torch.zeros((X.shape[0], W.shape[0])).half(),
             "gptq_rmsnorm_int8": lambda X, gamma, **kw: {"codes": X.char(), "xhat": X,
                                                          "scales": torch.ones(X.shape[0])},
             "gptq_regroup": lambda q, g_idx, *a: (q, g_idx),
             "gptq_packed_linear": lambda x, q, *a, **kw: torch.zeros((x.shape[0], q.shape[0])).half()}
    for name, f in fakes.items():
        monkeypatch.setattr(chain, name, watch(name, f))
    monkeypatch.setattr(chain, "_on", on, raising=False)

    class Torch:
        def __getattr__(self, name):
            return made(name, getattr(torch, name)) if name in ("zeros", "empty") else getattr(torch, name)

    monkeypatch.setattr(chain, "torch", Torch())
    X, Ws = torch.zeros((8, 64)).half(), [torch.zeros((96, 64)), torch.zeros((32, 96))]
    norms = [torch.ones(64).half(), torch.ones(96).half()] if normed else None
    chain.quantize_chain(X, Ws, bits=4, group=32, act_order=True, norms=norms, stream=given)
    assert not outside, outside


def test_regroup_reads_the_order_with_ordinary_loads():
    # The rows' kernels start while the order's kernel writes perm.  A load that asks
    # for data that nothing writes while the kernel lives (__ldg, or a const
    # __restrict__ pointer) may be taken from a stale line or moved before the wait.
    src = code_of("regroup.cu")
    kernels = re.findall(r"__global__.*?\n}\n", src, flags=re.S)
    readers = [k for k in kernels if "griddepcontrol.wait" in k]
    assert len(readers) == 2
    for k in readers:
        assert "const int32_t *perm" in k
        assert not re.search(r"__restrict__\s*perm\b", k)
        assert not re.search(r"__ld\w+\(\s*perm", k)
        assert not re.search(r"\bperm\b", k.split("{", 1)[1].split("griddepcontrol.wait")[0])


# ------------------------------------------------------------------ arguments that share memory
# Addresses far apart that are never dereferenced: each call below is refused before any
# CUDA call.

def apart(k, offset=0):
    return ctypes.c_void_p((1 << 40) * (k + 1) + offset)


def test_rmsnorm_refuses_shared_memory(lib):
    n, d = 4, 64
    names = ("x", "residual", "gamma", "perm", "h", "codes", "scales", "xhat")
    size = {"x": n * d * 2, "residual": n * d * 2, "gamma": d * 2, "perm": d * 4, "h": n * d * 2,
            "codes": n * d, "scales": n * 4, "xhat": n * d * 2}

    def call(**kw):
        a = {k: kw.get(k, apart(i)) for i, k in enumerate(names)}
        return lib.gptq_rmsnorm_int8(a["x"], a["residual"], a["gamma"], 0, n, d, 1e-5, a["perm"], a["h"],
                                     a["codes"], a["scales"], a["xhat"], None)
    for out in ("h", "codes", "scales", "xhat"):
        for other in names:
            if other == out:
                continue
            last = (size[other] - 1) // 16 * 16           # shares the other's last bytes
            offsets = {0, last} if out != "h" or other not in ("x", "residual") else {16, last}
            for offset in offsets:
                assert call(**{out: apart(names.index(other), offset)}) == 1, (out, other, offset)


def test_packed_linear_refuses_shared_memory(lib):
    n, r, d, bits, group = 20, 8, 128, 4, 64
    names = ("x", "xs", "q", "s", "z", "perm", "bias", "y", "ws")
    need = lib.gptq_packed_linear_workspace_bytes(n, r, d, bits, group, 3, 1)
    size = {"x": n * d, "xs": n * 4, "q": r * d * bits // 8, "s": r * 2 * 4, "z": r * 2 * 4, "perm": d * 4,
            "bias": r * 2, "y": n * r * 2, "ws": need}
    assert need >= n * d * 2

    def call(**kw):
        a = {k: kw.get(k, apart(i)) for i, k in enumerate(names)}
        return lib.gptq_packed_linear(a["x"], 3, a["xs"], n, a["q"], a["s"], a["z"], a["perm"], r, d, bits,
                                      group, a["bias"], a["y"], 0, a["ws"], need, None)
    for other in names:
        if other != "y":
            for offset in {0, (size[other] - 1) // 16 * 16}:
                assert call(y=apart(names.index(other), offset)) == 1, ("y", other, offset)
        if other != "ws":
            assert call(ws=apart(names.index(other))) == 1, ("ws", other)


def test_regroup_refuses_shared_memory(lib):
    r, d, bits, group = 4, 128, 4, 64
    names = ("q", "g_idx", "out", "perm")
    size = {"q": r * d * bits // 8, "g_idx": d * 4, "out": r * d * bits // 8, "perm": d * 4}

    def call(**kw):
        a = {k: kw.get(k, apart(i)) for i, k in enumerate(names)}
        return lib.gptq_regroup(a["q"], a["g_idx"], r, d, bits, group, a["out"], a["perm"], None)
    for mine in ("out", "perm"):
        for other in names:
            if other != mine:
                for offset in (0, size[other] - 4):
                    assert call(**{mine: apart(names.index(other), offset)}) == 1, (mine, other, offset)
