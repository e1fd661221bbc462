"""The operators of the 8-bit feed-forward block, as cases to time and to compare.

Kinds of case:
  weights     a packed layer with one scale per row laid out as 8-bit integers
  linear      y = x W^T (+ bias), 8-bit integers with a scale per token and per row of W
  gated       y = act(x G^T) * (x U^T), both products in 8-bit integers
  activation  act(x) (* up) in symmetric 8-bit codes with one scale per token

`run` computes a case with elementary torch operations, or with the package's
entry points when `own` is true.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the widest layers of the benchmark's 4096-wide block and of its 8192-wide one, laid out once
        _weights("weights_up", 11008, 4096, 8),
        _weights("weights_3bit", 8192, 8192, 3),
        # one new token through a square attention projection: latency
        _linear("linear_token", 1, 4096, 4096, "bf16"),
        # a batch of decoding sequences through a down projection
        _linear("linear_batch", 24, 4096, 11008, "fp16", bias=True),
        # one new token through the widest layer of the benchmark: HBM traffic
        _linear("linear_token_wide", 1, 12288, 49152, "fp16"),
        # a prompt through the down projection: tensor cores
        _linear("linear_prompt", 4096, 4096, 11008, "bf16"),
        # one new token through the gate and up projections
        _gated("gated_token", 1, 11008, 4096, "bf16", "silu"),
        # a ragged batch of short prompts
        _gated("gated_ragged", 333, 11008, 4096, "fp16", "gelu"),
        # a prompt: tensor cores
        _gated("gated_prompt", 4096, 11008, 4096, "bf16", "silu"),
        # one new token in front of the down projection: latency
        _activation("activation_token", 1, 11008, "bf16", "silu", True),
        # tokens of the widest layer of the benchmark, which has relu and no gate
        _activation("activation_relu", 500, 49152, "fp16", "relu", False),
        # a prompt with gate and up from products of fewer bits: HBM traffic
        _activation("activation_prompt", 4096, 11008, "bf16", "silu", True),
    ]


def _weights(name, r, d, bits):
    return {"name": name, "kind": "weights", "r": r, "d": d, "bits": bits}


def _linear(name, n, r, d, dtype, bias=False):
    return {"name": name, "kind": "linear", "n": n, "r": r, "d": d, "dtype": dtype, "bias": bias}


def _gated(name, n, r, d, dtype, act, bias=False):
    return {"name": name, "kind": "gated", "n": n, "r": r, "d": d, "dtype": dtype, "act": act, "bias": bias}


def _activation(name, n, d, dtype, act, gated):
    return {"name": name, "kind": "activation", "n": n, "d": d, "dtype": dtype, "act": act, "gated": gated}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["weights", "linear", "linear", "linear", "gated", "gated", "activation", "activation"])
    acts = ["silu", "silu", "gelu", "relu", "none"]
    if kind == "activation":
        n, d = log(1, 4096), 32 * log(2, 1536)
        n = max(1, min(n, 4096 * 11008 // d))
        c = _activation("", n, d, rng.choice(["fp16", "bf16"]), rng.choice(acts), rng.random() < 0.6)
    else:
        d = 32 * log(2, 1536)
        r = min(log(33, 16384), 12288 * 49152 // d)
        if kind == "weights":
            c = _weights("", max(1, min(r, 8192 * 8192 // d)), d, rng.choice([2, 3, 4, 8, 8]))
        elif kind == "linear":
            n = max(1, min(log(1, 4096), 4096 * 4096 * 11008 // (r * d)))
            c = _linear("", n, r, d, rng.choice(["fp16", "bf16", "bf16", "fp32"]), rng.random() < 0.3)
        else:
            r = min(r, 12288 * 49152 // (2 * d))
            n = max(1, min(log(1, 4096), 4096 * 4096 * 11008 // (r * d)))
            c = _gated("", n, r, d, rng.choice(["fp16", "bf16", "bf16", "fp32"]), rng.choice(acts), rng.random() < 0.2)
    del c["name"]
    return c


def work(case):
    d = case["d"]
    if case["kind"] == "weights":
        r = case["r"]
        # words, scales and zero points in; values and scales out
        return {"bytes": r * d * case["bits"] // 8 + 8 * r + r * d + 4 * r, "flops": r * d}
    n = case["n"]
    if case["kind"] == "activation":
        # x (and up) in; codes, their values in 16 bits and scales out
        return {"bytes": n * d * (7 if case["gated"] else 5) + 4 * n, "flops": 10 * n * d}
    r, size = case["r"], 4 if case["dtype"] == "fp32" else 2
    both = 2 if case["kind"] == "gated" else 1
    layer = r * d + 4 * r + (size * r if case["bias"] else 0)
    return {"bytes": both * layer + n * d + 4 * n + size * n * r, "flops": both * 2 * n * r * d}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    d, kind = case["d"], case["kind"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if kind == "weights":
        r, bits = case["r"], case["bits"]
        # every bit pattern is a valid row of codes
        s["qweight"] = torch.randint(-2 ** 31, 2 ** 31, (r, d * bits // 32), generator=gen, device=dev,
                                     dtype=torch.int64).to(torch.int32)
        s["scales"] = torch.exp(0.3 * normal(r, 1)) * (0.08 / (2 ** bits - 1))
        # 8 bits: the symmetric quantiser's zero point
        s["zeros"] = torch.full((r, 1), 128, device=dev, dtype=torch.int32) if bits == 8 else \
            torch.randint(0, 2 ** bits, (r, 1), generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
        s["w"] = torch.empty((r, d), dtype=torch.int8, device=dev)
        s["w_scales"] = torch.empty(r, dtype=torch.float32, device=dev)
        return s
    n, T = case["n"], DTYPES[case["dtype"]]
    if kind == "activation":
        # channels of different strength, a few far out, as in front of a down projection
        channel = torch.exp(0.7 * normal(d))
        channel[torch.randint(0, d, (max(1, d // 1000),), generator=gen, device=dev)] *= 8
        s["x"] = (normal(n, d) * channel).to(T)
        s["up"] = (normal(n, d) * channel).to(T) if case["gated"] else None
        s["outputs"] = {"codes": torch.empty((n, d), dtype=torch.int8, device=dev),
                        "scales": torch.empty(n, dtype=torch.float32, device=dev),
                        "xhat": torch.empty((n, d), dtype=T, device=dev)}
        return s
    r = case["r"]
    channel = torch.exp(0.7 * normal(d))
    channel[torch.randint(0, d, (max(1, d // 1000),), generator=gen, device=dev)] *= 30
    s["x"], s["x_scales"] = _codes(normal(n, d) * channel)
    # rows of the symmetric quantiser whose products with x are of order one
    for k in ("w", "up") if kind == "gated" else ("w",):
        w = torch.empty((r, d), dtype=torch.int8, device=dev)
        scales = torch.empty(r, dtype=torch.float32, device=dev)
        each = max(1, (1 << 26) // d)
        for a in range(0, r, each):
            w[a:a + each], scales[a:a + each] = _codes(normal(min(each, r - a), d) / math.sqrt(3 * d))
        s[k], s[k + "_scales"] = w, scales
        s[k + "_bias"] = (0.5 * normal(r)).to(T) if case["bias"] else None
    s["y"] = torch.empty((n, r), dtype=T, device=dev)
    return s


def _codes(x):
    scale = x.abs().amax(1) / 127
    return (x / scale[:, None]).round().clamp(-128, 127).to(torch.int8), scale


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import post_weight_quantization_19_b200 as g

        if kind == "weights":
            w, scales = g.gptq_int8_weights(s["qweight"], s["scales"], s["zeros"], case["d"], case["bits"],
                                            w=s["w"], w_scales=s["w_scales"])
            return {"w": w, "scales": scales}
        if kind == "linear":
            return g.gptq_int8_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], bias=s["w_bias"], y=s["y"])
        if kind == "gated":
            return g.gptq_int8_gated(s["x"], s["x_scales"], s["w"], s["w_scales"], s["up"], s["up_scales"],
                                     activation=case["act"], gate_bias=s["w_bias"], up_bias=s["up_bias"], y=s["y"])
        res = g.gptq_activation_int8(s["x"], s["up"], activation=case["act"], outputs=s["outputs"])
        return {k: v for k, v in res.items() if k != "codes"}
    if kind == "weights":
        q = _unpack(s["qweight"], case["bits"], case["d"])
        return {"w": (q - s["zeros"]).to(torch.int8), "scales": s["scales"][:, 0].clone()}
    if kind == "linear":
        return _plain_linear(s, "w").to(s["y"].dtype)
    if kind == "gated":
        return (_act(_plain_linear(s, "w"), case["act"]) * _plain_linear(s, "up")).to(s["y"].dtype)
    return _plain_activation(s)


def _unpack(qweight, bits, d):
    # code c sits at stream bits [c bits, (c + 1) bits) of its row, low bits first
    pos = torch.arange(d, device=qweight.device) * bits
    word, off = pos // 32, (pos % 32).to(torch.int32)
    inside = torch.clamp(32 - off, max=bits)
    low = (qweight[:, word] >> off) & ((1 << inside) - 1)
    if 32 % bits == 0:
        return low
    high = qweight[:, torch.clamp(word + 1, max=qweight.shape[1] - 1)]
    return low | ((high & ((1 << (bits - inside)) - 1)) << inside)


def _plain_linear(s, k):
    y = (s["x"].float() @ s[k].float().t()) * s["x_scales"][:, None] * s[k + "_scales"]
    return y if s[k + "_bias"] is None else y + s[k + "_bias"].float()


def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(v * -math.sqrt(0.5))
    return v


def _plain_activation(s):
    case = s["case"]
    # in 64 bits: a code next to a rounding border turns on the last bits
    u = _act(s["x"].double(), case["act"])
    if s["up"] is not None:
        u = u * s["up"].double()
    top = u.abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, torch.round(127 * u / top), torch.zeros_like(u))
    scale = torch.where(top > 0, top / 127, torch.ones_like(top)).float()
    return {"scales": scale[:, 0], "xhat": (codes.float() * scale).to(s["x"].dtype)}


def exact(case, seed):
    s = prepare(case, seed)
    f64, kind = torch.float64, case["kind"]
    if kind == "weights":
        return None
    if kind == "activation":
        v = s["x"].to(f64)
        u = _act64(v, case["act"])
        if case["gated"]:
            u = s["up"].to(f64) * u
        top = torch.maximum(u.max(1).values, -u.min(1).values)[:, None]
        empty = top == 0
        codes = (u * 127).div(torch.where(empty, torch.ones_like(top), top)).round()
        scale = torch.where(empty, torch.ones_like(top), top / 127)
        return {"scales": scale[:, 0], "xhat": codes * scale}
    out = []
    for k in ("w", "up") if kind == "gated" else ("w",):
        v = torch.empty((case["n"], case["r"]), dtype=f64, device=s["x"].device)
        each = max(1, (1 << 26) // case["d"])
        for a in range(0, case["r"], each):
            rows = s[k][a:a + each].to(f64) * s[k + "_scales"][a:a + each, None].to(f64)
            v[:, a:a + each] = torch.einsum("td,rd->tr", s["x"].to(f64) * s["x_scales"][:, None].to(f64), rows)
        if case["bias"]:
            v = v + s[k + "_bias"].to(f64)
        out.append(v)
    return out[0] if kind == "linear" else _act64(out[0], case["act"]) * out[1]


def _act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return v
