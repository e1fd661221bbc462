"""The operators that use a packed layer, as cases to time and to compare.

Kinds of case:
  norm     residual add + RMS norm + symmetric 8-bit codes with one scale per token
  linear   y = x W^^T (+ bias) from the packed layer, 16-bit activations
  linear8  the same from 8-bit activations with one scale per token
  regroup  the columns of an act-order layer sorted by group, with the order

`run` computes a case with elementary torch operations, or with the package's
entry points when `own` is true.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token through a 4096-wide block: latency of the norm
        _norm("norm_token", 1, 4096, "bf16", True),
        # a ragged batch of the widest activation of the 4096 model (no residual before its down projection)
        _norm("norm_ragged", 333, 11008, "fp16", False),
        # a prompt through the norm: HBM traffic
        _norm("norm_prompt", 4096, 4096, "bf16", True),
        # one new token through a square attention projection
        _linear("linear_token", 1, 4096, 4096, 4, 128, "fp16", False),
        # one new token through the widest layer of the benchmark, 3 bits: HBM traffic
        _linear("linear_token_wide", 1, 12288, 49152, 3, 128, "bf16", False),
        # a batch of decoding sequences through an act-order down projection
        _linear("linear_batch_actorder", 24, 4096, 11008, 4, 128, "fp16", True),
        # a prompt through the down projection: tensor cores
        _linear("linear_prompt", 4096, 4096, 11008, 4, 128, "bf16", False),
        # one new token with 8-bit activations
        _linear8("linear8_token", 1, 11008, 4096, 4, 128, "fp16"),
        # a small batch, 3-bit weights with one scale per row
        _linear8("linear8_batch", 8, 8192, 8192, 3, -1, "bf16"),
        # a ragged prompt with 8-bit activations
        _linear8("linear8_prompt", 1000, 11008, 4096, 4, 128, "bf16"),
        # the act-order layers of the benchmark, laid out once for the products
        _regroup("regroup_up", 11008, 4096, 4, 128),
        _regroup("regroup_wide", 8192, 8192, 3, 128),
    ]


def _norm(name, n, d, dtype, residual):
    return {"name": name, "kind": "norm", "n": n, "d": d, "dtype": dtype, "residual": residual}


def _linear(name, n, r, d, bits, group, dtype, actorder, bias=False):
    return {"name": name, "kind": "linear", "n": n, "r": r, "d": d, "bits": bits, "group": group,
            "dtype": dtype, "actorder": actorder, "bias": bias}


def _linear8(name, n, r, d, bits, group, dtype, bias=False):
    return {"name": name, "kind": "linear8", "n": n, "r": r, "d": d, "bits": bits, "group": group,
            "dtype": dtype, "actorder": False, "bias": bias}


def _regroup(name, r, d, bits, group):
    return {"name": name, "kind": "regroup", "r": r, "d": d, "bits": bits, "group": group}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["norm", "linear", "linear", "linear8", "linear8", "regroup"])
    dtype = rng.choice(["fp16", "bf16"])
    if kind == "norm":
        n, d = log(1, 4096), 32 * log(2, 1536)
        n = max(1, min(n, 4096 * 4096 // d))
        c = _norm("", n, d, dtype, rng.random() < 0.6)
    else:
        bits = rng.choice([2, 3, 4, 4, 4, 8])
        group = rng.choice([-1, 32, 64, 96, 128, 128, 128])
        step = 32 if group == -1 else group
        d = step * max(1, log(64, 49152) // step)
        r = min(log(33, 16384), 12288 * 49152 // d)
        if kind == "regroup":
            group = 128 if group == -1 else group
            d = group * max(2, d // group)
            r = max(1, min(r, 8192 * 8192 // d))
            c = _regroup("", r, d, bits, group)
        else:
            n = max(1, min(log(1, 4096), 4096 * 4096 * 11008 // (r * d)))
            make = _linear8 if kind == "linear8" else _linear
            more = {} if kind == "linear8" else {"actorder": group > 0 and rng.random() < 0.3}
            c = make("", n, r, d, bits, group, dtype, bias=rng.random() < 0.3, **more)
    del c["name"]
    return c


def work(case):
    d = case["d"]
    if case["kind"] == "norm":
        n = case["n"]
        # x (and the residual) in; codes, their values in 16 bits, scales (and the sum) out
        per = 2 + 1 + 2 + (4 if case["residual"] else 0)
        return {"bytes": n * d * per + 2 * d + 4 * n, "flops": 10 * n * d}
    codes = case["r"] * d * case["bits"] // 8
    if case["kind"] == "regroup":
        return {"bytes": 2 * codes + 8 * d, "flops": 0}
    n, r, groups = case["n"], case["r"], _groups(case)
    x = n * d * 2 if case["kind"] == "linear" else n * d + 4 * n
    more = (4 * d if case["actorder"] else 0) + (2 * r if case["bias"] else 0)
    return {"bytes": codes + 8 * r * groups + x + 2 * n * r + more, "flops": 2 * n * r * d}


def _groups(case):
    return 1 if case["group"] == -1 else case["d"] // case["group"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    d = case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def words(r):
        # every bit pattern is a valid row of codes
        return torch.randint(-2 ** 31, 2 ** 31, (r, d * case["bits"] // 32), generator=gen,
                             device=dev, dtype=torch.int64).to(torch.int32)

    s = {"case": case}
    if case["kind"] == "regroup":
        s["qweight"] = words(case["r"])
        order = torch.randperm(d, generator=gen, device=dev)
        s["g_idx"] = torch.empty(d, dtype=torch.int32, device=dev)
        s["g_idx"][order] = (torch.arange(d, device=dev) // case["group"]).to(torch.int32)
        s["out"] = torch.empty_like(s["qweight"])
        s["perm"] = torch.empty_like(s["g_idx"])
        return s
    n, T = case["n"], DTYPES[case["dtype"]]
    # channels of different strength with a few outliers, as calibration activations have
    channel = torch.exp(0.7 * normal(d))
    channel[torch.randint(0, d, (max(1, d // 1000),), generator=gen, device=dev)] *= 30
    if case["kind"] == "norm":
        s["x"] = (normal(n, d) * channel).to(T)
        s["gamma"] = (1 + 0.2 * normal(d)).to(T)
        s["residual"] = (normal(n, d) * channel).to(T) if case["residual"] else None
        s["outputs"] = {"codes": torch.empty((n, d), dtype=torch.int8, device=dev),
                        "scales": torch.empty(n, dtype=torch.float32, device=dev),
                        "xhat": torch.empty((n, d), dtype=T, device=dev)}
        if case["residual"]:
            s["outputs"]["h"] = torch.empty((n, d), dtype=T, device=dev)
        return s
    r, G = case["r"], _groups(case)
    top = 2 ** case["bits"] - 1
    s["qweight"] = words(r)
    s["scales"] = torch.exp(0.3 * normal(r, G)) * (0.08 / top)
    s["zeros"] = (0.5 * top + 0.1 * top * normal(r, G)).round().clamp(0, top).to(torch.int32)
    s["bias"] = normal(r).to(T) if case["bias"] else None
    s["perm"] = torch.randperm(d, generator=gen, device=dev).to(torch.int32) if case["actorder"] else None
    x = normal(n, d) * channel
    if case["kind"] == "linear":
        s["x"], s["x_scales"] = x.to(T), None
    else:
        s["x_scales"] = x.abs().amax(1) / 127
        s["x"] = (x / s["x_scales"][:, None]).round().clamp(-128, 127).to(torch.int8)
    s["y"] = torch.empty((n, r), dtype=T, device=dev)
    return s


def run(s):
    case = s["case"]
    if own:
        import post_weight_quantization_19_b200 as g

        if case["kind"] == "norm":
            res = g.gptq_rmsnorm_int8(s["x"], s["gamma"], eps=EPS, residual=s["residual"],
                                      outputs=s["outputs"])
            return {k: v for k, v in res.items() if k != "codes"}
        if case["kind"] == "regroup":
            q, perm = g.gptq_regroup(s["qweight"], s["g_idx"], case["bits"], case["group"],
                                     out=s["out"], perm=s["perm"])
            return {"qweight": q, "perm": perm}
        return g.gptq_packed_linear(s["x"], s["qweight"], s["scales"], s["zeros"], case["bits"],
                                    case["group"], x_scales=s["x_scales"], bias=s["bias"],
                                    perm=s["perm"], y=s["y"])
    if case["kind"] == "norm":
        return _plain_norm(s)
    if case["kind"] == "regroup":
        return _plain_regroup(s)
    return _plain_linear(s)


def _plain_norm(s):
    T = s["x"].dtype
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(T)
    # in 64 bits: a code next to a rounding border turns on the last bits
    u = h.double()
    u = u / torch.sqrt((u * u).mean(1, keepdim=True) + EPS) * s["gamma"].double()
    top = u.abs().amax(1, keepdim=True)
    scale = torch.where(top > 0, top / 127, torch.ones_like(top))
    codes = torch.clamp(torch.round(u / scale), -128, 127)
    scale = scale.float()
    out = {"scales": scale[:, 0], "xhat": (codes.float() * scale).to(T)}
    if s["residual"] is not None:
        out["h"] = h
    return out


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


def _plain_linear(s):
    case = s["case"]
    n, d, G = case["n"], case["d"], _groups(case)
    w = _unpack(s["qweight"], case["bits"], d).float().view(case["r"], G, d // G)
    w = ((w - s["zeros"].float()[:, :, None]) * s["scales"][:, :, None]).view(case["r"], d)
    x = s["x"].float()
    if s["x_scales"] is not None:
        x = x * s["x_scales"][:, None]
    if s["perm"] is not None:
        x = x[:, s["perm"].long()]
    y = x @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["y"].dtype)


def _plain_regroup(s):
    case = s["case"]
    d, bits = case["d"], case["bits"]
    perm = torch.sort(s["g_idx"], stable=True)[1]
    q = _unpack(s["qweight"], bits, d)[:, perm].view(case["r"], d // 32, 32)
    # 32 codes fill `bits` words: word k holds the parts of the codes inside stream bits [32 k, 32 k + 32)
    pos = torch.arange(32, device=q.device) * bits
    at = pos[:, None] - 32 * torch.arange(bits, device=q.device)[None, :]
    parts = torch.where(at >= 0, q.long()[..., None] << torch.clamp(at, 0, 32),
                        q.long()[..., None] >> torch.clamp(-at, 0, 32))
    full = (parts & 0xFFFFFFFF).sum(2)
    full = torch.where(full >= 2 ** 31, full - 2 ** 32, full)
    return {"qweight": full.to(torch.int32).view(case["r"], -1), "perm": perm.to(torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "regroup":
        return None
    f64 = torch.float64
    if case["kind"] == "norm":
        T = s["x"].dtype
        h = s["x"]
        if case["residual"]:
            h = (h.to(f64) + s["residual"].to(f64)).to(T)
        v = h.to(f64)
        u = s["gamma"].to(f64) * v * (v.square().sum(1) / case["d"] + EPS).rsqrt()[:, None]
        scale = u.abs().max(1).values / 127
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        codes = torch.round(u / scale[:, None]).clamp(-128, 127)
        out = {"scales": scale, "xhat": codes * scale[:, None]}
        if case["residual"]:
            out["h"] = None
        return out
    r, d, bits, group = case["r"], case["d"], case["bits"], case["group"]
    x = s["x"].to(f64)
    if case["kind"] == "linear8":
        x = x * s["x_scales"].to(f64)[:, None]
    if case["actorder"]:
        x = x.index_select(1, s["perm"].long())
    size = d if group == -1 else group
    y = torch.empty((case["n"], r), dtype=f64, device=x.device)
    each = max(1, (1 << 26) // d)
    for a in range(0, r, each):
        b = min(r, a + each)
        bit = (s["qweight"][a:b, :, None] >> torch.arange(32, dtype=torch.int32, device=x.device)) & 1
        bit = bit.reshape(b - a, d, bits).to(f64)
        q = (bit * (2.0 ** torch.arange(bits, dtype=f64, device=x.device))).sum(2)
        z = torch.repeat_interleave(s["zeros"][a:b].to(f64), size, dim=1)
        step = torch.repeat_interleave(s["scales"][a:b].to(f64), size, dim=1)
        y[:, a:b] = x @ ((q - z) * step).t()
    if case["bias"]:
        y = y + s["bias"].to(f64)
    return y
