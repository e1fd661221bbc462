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
