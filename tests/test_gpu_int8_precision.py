"""How exact the 8-bit block's activations are, where their values are small or near a border.

Tolerances from the arithmetic of each form, as the header states it; E is half a step of fp32
relative to the value.
"""

import numpy as np
import pytest

import oracle
from test_gpu_int8 import BF16, E, F16, F32, HALF, I8, f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def gated_of(gates, ups, act, T):
    """act(gate) up through gptq_int8_gated, gates and ups as they are: x and both layers are ones
    in their first column and zeros behind it, so that the sums are the rows' scales."""
    import post_weight_quantization_19_b200 as g
    r, d = gates.numel(), 32
    x = torch.zeros((1, d), dtype=I8, device="cuda")
    w = torch.zeros((r, d), dtype=I8, device="cuda")
    x[:, 0] = w[:, 0] = 1
    return g.gptq_int8_gated(x, torch.ones(1, device="cuda"), w, gates, w, ups, activation=act, dtype=T)[0]


def tail_gates(act):
    """Gates far below zero, down to values that fp32 holds with few digits or not at all."""
    low = {"silu": -104.0, "gelu": -14.5}[act]
    return torch.linspace(low, low / 2, 5001, dtype=torch.float64).float().cuda()


@pytest.mark.parametrize("up", [1.0, -3e5, 2.0 ** 100])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_fp32_of_gates_far_below_zero(act, up):
    # act within 6e-7 of its value (gelu: 1e-7 g^2 more), one rounding of the product; what
    # fp32 holds below its normal numbers: exp or erfc within two of its steps of 2^-149 there,
    # times |g|, and the products' own rounding to such a step
    gates = tail_gates(act)
    y = f64(gated_of(gates, torch.full_like(gates, up), act, F32))
    g = f64(gates)
    f = oracle.activation(g, act)
    own = 6e-7 + (1e-7 * g ** 2 if act == "gelu" else 0.0)
    tol = (own * np.abs(f) + 3e-43) * abs(up) + E * np.abs(f * up) + 2.0 ** -149
    assert np.all(np.abs(y - f * up) <= tol), (np.abs(y - f * up) / tol).max()


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_16_bit_of_gates_far_below_zero(act, T):
    # the same, values below 1e-35 lost; times 2^100, where bf16 tells them
    gates = tail_gates(act)
    for up in (1.0, 2.0 ** 100) if T == BF16 else (1.0, 2.0 ** 30):
        y = f64(gated_of(gates, torch.full_like(gates, up), act, T))
        g = f64(gates)
        f = oracle.activation(g, act)
        own = 6e-7 + (1e-7 * g ** 2 if act == "gelu" else 0.0)
        tol = (own * np.abs(f) + 1e-35) * up + (HALF[T] * (1 + 1e-5) + E) * np.abs(f * up)
        tol = tol + (2.0 ** -25 if T == F16 else 0.0)
        assert np.all(np.abs(y - f * up) <= tol), (np.abs(y - f * up) / tol).max()


def selftest(lib, v, act):
    n = v.numel()
    values = torch.empty((3, n), device="cuda")
    values64 = torch.empty(n, dtype=torch.float64, device="cuda")
    which = ["none", "relu", "silu", "gelu"].index(act)
    assert lib.gptq_selftest_activation(v.data_ptr(), n, which, values.data_ptr(), values64.data_ptr(),
                                        torch.cuda.current_stream().cuda_stream) == 0
    return (*(f64(t) for t in values), f64(values64))


def off(got, want, relative, lost):
    """The largest part of its tolerance that a value is off by (NaN counts as off)."""
    with np.errstate(invalid="ignore", over="ignore"):
        return float(np.nan_to_num(np.abs(got - want) / (relative * np.abs(want) + lost), nan=np.inf).max())


@pytest.mark.parametrize("T", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_of_every_16_bit_number(lib, act, T):
    # What the codes of gptq_activation_int8 rest on: values in fp32 within 4.3e-7, less than what
    # decides which ones are formed again (1e-6, with the product's rounding), and those within
    # 1e-13.  Only values that are not coded as 0 are formed again: with a row's largest 1e-22
    # at least and up 1e6 at most, 1e-22 / 254 / 1e6 = 3.9e-31 at least.  The oracle's own error, in 64 bits: exp and erfc to a few 2^-53, erfc's
    # argument to half a step, worth v^2 2^-53 of the value.
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(T)
    v = v[torch.isfinite(v)].float().cuda()
    want = oracle.activation(f64(v), act)
    exact, whole, fast, single = selftest(lib, v, act)
    size = np.abs(f64(v))
    assert off(whole, want, 4.3e-7, 1e-35) <= 1
    # (beyond these the row is done in 64 bits: a NaN, or an infinity, leaves its safe range)
    inside = size < (2.3e38 if act == "silu" else 1e19)
    assert off(fast[inside], want[inside], 4.3e-7, 1e-35) <= 1
    tops = np.abs(fast[~inside])
    assert np.all(np.isnan(tops) | (tops > 1e18) | (want[~inside] == 0))
    squares = np.minimum(size, 40.0) ** 2
    assert off(exact, want, 6e-7 + (1e-7 * squares if act == "gelu" else 0.0), 3e-43) <= 1
    asked = np.abs(want) >= 1e-31
    assert off(single[asked], want[asked], 1e-13 + 2.0 ** -53 * (8 + squares[asked]), 0.0) <= 1


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_of_fp32_numbers(lib, act):
    # The gated block's arguments, which are no numbers of 16 bits.  For its results of 16 bits, in
    # units of 1e-8 of the value: exp 24 (ex2's 2^-22) and 6 for the step to first order; silu: 6
    # for 1 + exp, 12 for the reciprocal (2^-23), 6 for the product, 54 in all.  gelu: 6 and 12
    # for t, whose share of the tail is at most as large; the polynomial's coefficients 7.1, its
    # nine steps 6 times what the later ones leave of each (1, .8, .6, .4, .3, .1, .3, .3, .1: 23);
    # exp 30; three products 18: 96 in all, and exp's argument -v^2 / 2, rounded, 3 v^2.
    rng = np.random.default_rng(1)
    v = np.concatenate([np.linspace(-110, 110, 2000001), np.linspace(-15, 15, 2000001),
                        rng.standard_normal(200000) * 10.0 ** rng.integers(-30, 38, 200000)])
    v = torch.from_numpy(v.astype(np.float32)).cuda()
    v = v[torch.isfinite(v)]
    want = oracle.activation(f64(v), act)
    exact, whole, _, single = selftest(lib, v, act)
    squares = np.minimum(np.abs(f64(v)), 40.0) ** 2
    gelu = act == "gelu"
    assert off(exact, want, 6e-7 + (1e-7 * squares if gelu else 0.0), 3e-43) <= 1
    assert off(whole, want, 9.7e-7 + 3.1e-8 * squares if gelu else 5.5e-7, 1e-35) <= 1
    asked = np.abs(want) >= 1e-31
    assert off(single[asked], want[asked], 1e-13 + 2.0 ** -53 * (8 + squares[asked]), 0.0) <= 1


@pytest.mark.parametrize("act", ["none", "relu"])
def test_activations_that_round_nothing(lib, act):
    v = torch.randn(4099, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    want = oracle.activation(f64(v), act)
    for got in selftest(lib, v, act):
        np.testing.assert_array_equal(got, want)
