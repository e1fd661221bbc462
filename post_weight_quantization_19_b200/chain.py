"""A chain of linear layers quantised in order, each calibrated on the outputs
of the quantised layers before it.

GPTQ reading card, §计算设置: the reference implementation loads one block at a
time, accumulates the layer Hessians, quantises the block, then runs the
quantised block to produce the next block's inputs.  Here the chain is a
sequence of linear layers with no nonlinearity between them: layer k is solved
on H_k = 2 X_k^T X_k, and X_{k+1} = fp16(X_k fp16(W^_k)^T) is computed from its
packed output (dequantised to FP16 and multiplied in floating point, as the
"GPTQ" concept page describes inference, §3 技術原理).  Every step runs in the
library's kernels: the Hessian, the solve, the FP16 dequantisation and the
forward product.

With ``norms``, a layer runs as it would be served with 8-bit activations: its
input is the root-mean-square norm of X_k in 8-bit codes with one scale per
token (``gptq_rmsnorm_int8``), H_k is that of the values the codes stand for, and
X_{k+1} comes from the codes and the packed weights (``gptq_packed_linear``;
act-order layers laid out by group first, ``gptq_regroup``).
"""

from __future__ import annotations

import torch

from .gptq import (_on, gptq_dequant_fp16, gptq_hessian_accumulate, gptq_linear_fp16,
                   gptq_packed_linear, gptq_quantize_layer, gptq_regroup, gptq_rmsnorm_int8)


def quantize_chain(X0: torch.Tensor, Ws: list, *, bits: int, group: int, block: int = 128,
                   damp: float = 0.01, act_order: bool = False, sym: bool = False,
                   static_groups: bool = False, keep_inputs: bool = False,
                   norms: list | None = None, eps: float = 1e-6, stream=None) -> list[dict]:
    """Quantise W_0, W_1, ... (fp32 [r_k, d_k], d_{k+1} = r_k) on calibration
    tokens X0 (fp16 [n, d_0]).

    Returns one ``gptq_quantize_layer`` result per layer (with ``g_idx``), plus
    ``inputs`` = X_k when ``keep_inputs``, and ``outputs`` = X_{k+1} for the last
    layer.  The tensors stay on the device and belong to ``stream`` (the current
    one by default), which X0, Ws and the norms must be ready on.  The host waits
    for a layer's solve, which reads its loss back, and in an act-order layer with
    a norm for the check of its order (``gptq_regroup``).

    ``norms`` holds gamma (fp16 [d_k]) for each layer whose input is normed and
    held in 8 bits, None for the others; ``eps`` is the norms' own.  Such a layer's
    result also has ``in_codes`` and ``in_scales``, and for an act-order layer
    ``qweight_by_group`` and ``perm``; its ``inputs`` are the codes' values in fp16.
    """
    if norms is not None and len(norms) != len(Ws):
        raise ValueError(f"{len(norms)} norms for {len(Ws)} layers")
    with _on(stream):   # what is allocated and filled here belongs to the stream that uses it
        X = X0
        outs = []
        for k, W in enumerate(Ws):
            r, d = W.shape
            if X.shape[1] != d:
                raise ValueError(f"layer {k}: W has {d} inputs, the previous layer gives {X.shape[1]}")
            normed = None
            if norms is not None and norms[k] is not None:
                normed = gptq_rmsnorm_int8(X, norms[k], eps=eps, xhat=True, stream=stream)
                X = normed["xhat"]
            H = torch.zeros((d, d), dtype=torch.float32, device=W.device)
            gptq_hessian_accumulate(X, H, stream=stream)
            g_idx = torch.empty(d, dtype=torch.int32, device=W.device)
            res = gptq_quantize_layer(W, H, bits=bits, group=group, block=block, damp=damp,
                                      act_order=act_order, sym=sym, static_groups=static_groups,
                                      g_idx=g_idx, stream=stream)
            if keep_inputs:
                res["inputs"] = X
            if normed is None:
                W16 = gptq_dequant_fp16(res["qweight"], res["scales"], res["zeros"], d, bits, group,
                                        g_idx=g_idx, stream=stream)
                X = gptq_linear_fp16(X, W16, stream=stream)
            else:
                res["in_codes"], res["in_scales"] = normed["codes"], normed["scales"]
                qweight, perm = res["qweight"], None
                if act_order and group != -1 and not static_groups:   # else groups are contiguous
                    qweight, perm = gptq_regroup(qweight, g_idx, bits, group, stream=stream)
                    res["qweight_by_group"], res["perm"] = qweight, perm
                X = gptq_packed_linear(normed["codes"], qweight, res["scales"], res["zeros"], bits, group,
                                       x_scales=normed["scales"], perm=perm, stream=stream)
            outs.append(res)
        if outs:
            outs[-1]["outputs"] = X
    return outs
