"""Python binding of the C ABI: the same entry points, taking torch CUDA tensors.

Argument marshalling only -- dtype/shape/device checks and pointer extraction.
Every step of the solve runs in the CUDA kernels of libgptq_b200.so; there is
no CPU path.  PyTorch provides device memory and streams.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _abi


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _abi.load()
        msg = lib.gptq_status_string(status).decode()
        detail = lib.gptq_last_error().decode() if status == 3 else ""
        super().__init__(f"{where}: {_abi.STATUS.get(status, status)} ({msg})"
                         + (f": {detail}" if detail else ""))
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise GPTQError(status, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# Option bits of the layer solve (include/gptq.h).
ACT_ORDER, SYMMETRIC, STATIC_GROUPS = 1, 2, 4


def _options(act_order: bool, sym: bool, static_groups: bool) -> int:
    return ((ACT_ORDER if act_order else 0) | (SYMMETRIC if sym else 0)
            | (STATIC_GROUPS if static_groups else 0))


def _ptr(t: torch.Tensor | None, dtype: torch.dtype | None = None, name: str = "") -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def gptq_hessian_accumulate(X: torch.Tensor, H: torch.Tensor, stream=None) -> None:
    """H += 2 X^T X on the GPU (X fp16 [n, d] row-major, H fp32 [d, d])."""
    lib = _abi.load()
    n, d = X.shape
    if H.shape != (d, d):
        raise ValueError("H must be [d, d]")
    _check(lib.gptq_hessian_accumulate(_ptr(X, torch.float16, "X"), n, d, d,
                                       _ptr(H, torch.float32, "H"), _stream(stream)),
           "gptq_hessian_accumulate")


def gptq_quantize_workspace_bytes(r: int, d: int, bits: int, group: int, block: int = 128,
                                  act_order: bool = False, sym: bool = False,
                                  static_groups: bool = False) -> int:
    return int(_abi.load().gptq_quantize_workspace_bytes(
        r, d, bits, group, block, _options(act_order, sym, static_groups)))


def gptq_quantize_layer(W: torch.Tensor, H: torch.Tensor, *, bits: int, group: int,
                        block: int = 128, damp: float = 0.01, act_order: bool = False,
                        sym: bool = False, static_groups: bool = False,
                        W_hat: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                        g_idx: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        outputs: dict | None = None, stream=None) -> dict:
    """GPTQ solve of one layer.  H is consumed.  Returns qweight/scales/zeros/loss (+ optional).

    ``sym`` selects the symmetric quantiser and ``static_groups`` fixes every
    group's parameters from the original W before the sweep (GPTQ_SYMMETRIC and
    GPTQ_STATIC_GROUPS of the C header).  ``outputs`` may hold preallocated
    ``qweight``, ``scales`` and ``zeros`` tensors.
    """
    options = _options(act_order, sym, static_groups)
    lib = _abi.load()
    r, d = W.shape
    G = 1 if group == -1 else d // max(group, 1)
    dev = W.device
    out = dict(outputs or {})
    qweight = out.get("qweight")
    if qweight is None:
        qweight = torch.empty((r, d * bits // 32), dtype=torch.int32, device=dev)
    scales = out.get("scales")
    if scales is None:
        scales = torch.empty((r, G), dtype=torch.float32, device=dev)
    zeros = out.get("zeros")
    if zeros is None:
        zeros = torch.empty((r, G), dtype=torch.int32, device=dev)
    need = lib.gptq_quantize_workspace_bytes(r, d, bits, group, block, options)
    if need == 0 and r > 0:
        raise GPTQError(1, "gptq_quantize_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    loss = ctypes.c_double(0.0)
    _check(lib.gptq_quantize_layer(
        _ptr(W, torch.float32, "W"), r, d, _ptr(H, torch.float32, "H"), bits, group, block,
        float(damp), options, _ptr(W_hat, torch.float32, "W_hat"),
        _ptr(qweight, torch.int32, "qweight"), _ptr(scales, torch.float32, "scales"),
        _ptr(zeros, torch.int32, "zeros"), _ptr(g_idx, torch.int32, "g_idx"),
        _ptr(codes, torch.uint8, "codes"), ctypes.byref(loss), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "gptq_quantize_layer")
    res = {"qweight": qweight, "scales": scales, "zeros": zeros, "loss": loss.value}
    if W_hat is not None:
        res["W_hat"] = W_hat
    if codes is not None:
        res["codes"] = codes
    if g_idx is not None:
        res["g_idx"] = g_idx
    return res


def gptq_dequant_gemv(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                      x: torch.Tensor, bits: int, group: int, g_idx: torch.Tensor | None = None,
                      y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [m, r] = x [m, d] W^^T from the packed layer (x fp32, m <= GPTQ_GEMV_MAX_M)."""
    lib = _abi.load()
    if x.dim() == 1:
        x = x.unsqueeze(0)
    m, d = x.shape
    r = qweight.shape[0]
    if y is None:
        y = torch.empty((m, r), dtype=torch.float32, device=x.device)
    _check(lib.gptq_dequant_gemv(
        _ptr(qweight, torch.int32, "qweight"), _ptr(scales, torch.float32, "scales"),
        _ptr(zeros, torch.int32, "zeros"), _ptr(g_idx, torch.int32, "g_idx"), r, d, bits, group,
        _ptr(x, torch.float32, "x"), m, _ptr(y, torch.float32, "y"), _stream(stream)),
        "gptq_dequant_gemv")
    return y


def gptq_factor(H: torch.Tensor, *, damp: float = 0.01, act_order: bool = False,
                workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Damp, order and factor H in place: returns {"U": H, "perm", "lambda"} for
    ``gptq_quantize_with_factor`` (perm is None without act-order)."""
    lib = _abi.load()
    d = H.shape[0]
    if H.shape != (d, d):
        raise ValueError("H must be [d, d]")
    options = ACT_ORDER if act_order else 0
    need = lib.gptq_factor_workspace_bytes(d, options)
    if need == 0:
        raise GPTQError(1, "gptq_factor_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=H.device)
    perm = torch.empty(d, dtype=torch.int32, device=H.device) if act_order else None
    lam = torch.empty(1, dtype=torch.float32, device=H.device)
    _check(lib.gptq_factor(_ptr(H, torch.float32, "H"), d, float(damp), options,
                           _ptr(perm, torch.int32, "perm"), _ptr(lam, torch.float32, "lambda"),
                           _ptr(workspace, None, "workspace"),
                           workspace.numel() * workspace.element_size(), _stream(stream)),
           "gptq_factor")
    return {"U": H, "perm": perm, "lambda": lam}


def gptq_quantize_with_factor(W: torch.Tensor, factor: dict, *, bits: int, group: int,
                              block: int = 128, sym: bool = False, static_groups: bool = False,
                              W_hat: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                              g_idx: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, outputs: dict | None = None,
                              stream=None) -> dict:
    """The sweep half of the solve from ``gptq_factor``'s result (U, perm, lambda are
    only read).  Returns qweight/scales/zeros/loss like ``gptq_quantize_layer``."""
    lib = _abi.load()
    r, d = W.shape
    U, perm, lam = factor["U"], factor["perm"], factor["lambda"]
    options = _options(perm is not None, sym, static_groups)
    G = 1 if group == -1 else d // max(group, 1)
    dev = W.device
    out = dict(outputs or {})
    qweight = out.get("qweight")
    if qweight is None:
        qweight = torch.empty((r, d * bits // 32), dtype=torch.int32, device=dev)
    scales = out.get("scales")
    if scales is None:
        scales = torch.empty((r, G), dtype=torch.float32, device=dev)
    zeros = out.get("zeros")
    if zeros is None:
        zeros = torch.empty((r, G), dtype=torch.int32, device=dev)
    need = lib.gptq_quantize_with_factor_workspace_bytes(r, d, bits, group, block)
    if need == 0 and r > 0:
        raise GPTQError(1, "gptq_quantize_with_factor_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    loss = ctypes.c_double(0.0)
    _check(lib.gptq_quantize_with_factor(
        _ptr(W, torch.float32, "W"), r, d, _ptr(U, torch.float32, "U"),
        _ptr(perm, torch.int32, "perm"), _ptr(lam, torch.float32, "lambda"), bits, group, block,
        options, _ptr(W_hat, torch.float32, "W_hat"), _ptr(qweight, torch.int32, "qweight"),
        _ptr(scales, torch.float32, "scales"), _ptr(zeros, torch.int32, "zeros"),
        _ptr(g_idx, torch.int32, "g_idx"), _ptr(codes, torch.uint8, "codes"), ctypes.byref(loss),
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), "gptq_quantize_with_factor")
    res = {"qweight": qweight, "scales": scales, "zeros": zeros, "loss": loss.value}
    if W_hat is not None:
        res["W_hat"] = W_hat
    if codes is not None:
        res["codes"] = codes
    if g_idx is not None:
        res["g_idx"] = g_idx
    return res


def gptq_dequant_fp16(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, d: int,
                      bits: int, group: int, g_idx: torch.Tensor | None = None,
                      W16: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W16 [r, d] fp16 = s (q - z) from the packed layer."""
    lib = _abi.load()
    r = qweight.shape[0]
    if W16 is None:
        W16 = torch.empty((r, d), dtype=torch.float16, device=qweight.device)
    _check(lib.gptq_dequant_fp16(
        _ptr(qweight, torch.int32, "qweight"), _ptr(scales, torch.float32, "scales"),
        _ptr(zeros, torch.int32, "zeros"), _ptr(g_idx, torch.int32, "g_idx"), r, d, bits, group,
        _ptr(W16, torch.float16, "W16"), _stream(stream)), "gptq_dequant_fp16")
    return W16


def gptq_linear_fp16(X: torch.Tensor, W16: torch.Tensor, Y: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Y [n, r] = fp16(X [n, d] W16 [r, d]^T), fp32 accumulation on the tensor cores."""
    lib = _abi.load()
    n, d = X.shape
    r = W16.shape[0]
    if W16.shape[1] != d:
        raise ValueError("W16 must be [r, d]")
    if Y is None:
        Y = torch.empty((n, r), dtype=torch.float16, device=X.device)
    _check(lib.gptq_linear_fp16(_ptr(X, torch.float16, "X"), n, d, _ptr(W16, torch.float16, "W16"),
                                r, _ptr(Y, torch.float16, "Y"), _stream(stream)),
           "gptq_linear_fp16")
    return Y


# Types of activations (include/gptq.h).
_DTYPE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.int8: 3}


def _shaped(t: torch.Tensor | None, dtype: torch.dtype, shape: tuple, device: torch.device,
            name: str) -> int | None:
    """Pointer of a contiguous tensor of this type, shape and device (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _activations(x: torch.Tensor, dtypes: tuple, name: str = "x") -> None:
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must be [tokens, features]")
    if x.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(map(str, dtypes))}, got {x.dtype}")


# The current device's index and its current stream's handle, without building
# torch's device and stream objects (about 2 us a call) where torch offers that.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(device: torch.device, stream, fn, *args) -> int:
    """fn(*args, stream) with the tensors' device current; the stream is the
    given one or that device's current stream."""
    if stream is None:
        handle = _raw_stream(device.index)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    else:
        handle = stream.cuda_stream
    if _current_device() == device.index:
        return fn(*args, handle)
    with torch.cuda.device(device):
        return fn(*args, handle)


def _on(stream):
    """Where a call's own tensors are allocated: on the stream that it works on, so
    that their memory, freed, is not taken while that stream still uses it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def gptq_rmsnorm_int8(x: torch.Tensor, gamma: torch.Tensor, *, eps: float,
                      residual: torch.Tensor | None = None, perm: torch.Tensor | None = None,
                      xhat: bool = False, outputs: dict | None = None, stream=None) -> dict:
    """h = x + residual, its root-mean-square norm times gamma, in symmetric 8-bit
    codes with one scale per token.

    x, residual [n, d] and gamma [d] fp16 or bf16.  Returns ``codes`` int8
    [n, d], ``scales`` fp32 [n], ``h`` when there is a residual, and ``xhat`` =
    scales * codes in x's type when asked for.  ``perm`` (from ``gptq_regroup``)
    gives codes and xhat in that column order.  ``outputs`` may hold
    preallocated tensors of these names (an ``xhat`` or ``h`` among them is
    written; ``h`` may be x or residual).
    """
    lib = _abi.load()
    _activations(x, (torch.float16, torch.bfloat16))
    n, d = x.shape
    dev, T = x.device, x.dtype
    out = dict(outputs or {})
    codes, scales, xh, h = (out.get(k) for k in ("codes", "scales", "xhat", "h"))
    with _on(stream):
        if codes is None:
            codes = torch.empty((n, d), dtype=torch.int8, device=dev)
        if scales is None:
            scales = torch.empty(n, dtype=torch.float32, device=dev)
        if xh is None and xhat:
            xh = torch.empty((n, d), dtype=T, device=dev)
        if h is None and residual is not None:
            h = torch.empty((n, d), dtype=T, device=dev)
    _check(_launch(
        dev, stream, lib.gptq_rmsnorm_int8, _shaped(x, T, (n, d), dev, "x"),
        _shaped(residual, T, (n, d), dev, "residual"), _shaped(gamma, T, (d,), dev, "gamma"),
        _DTYPE[T], n, d, float(eps), _shaped(perm, torch.int32, (d,), dev, "perm"),
        _shaped(h, T, (n, d), dev, "h"), _shaped(codes, torch.int8, (n, d), dev, "codes"),
        _shaped(scales, torch.float32, (n,), dev, "scales"),
        _shaped(xh, T, (n, d), dev, "xhat")), "gptq_rmsnorm_int8")
    res = {"codes": codes, "scales": scales}
    if h is not None:
        res["h"] = h
    if xh is not None:
        res["xhat"] = xh
    return res


def gptq_packed_linear_workspace_bytes(n: int, r: int, d: int, bits: int, group: int, *,
                                       x_dtype: torch.dtype = torch.float16,
                                       permuted: bool = False) -> int:
    if x_dtype not in (torch.float16, torch.bfloat16, torch.int8):
        raise ValueError(f"x must be float16, bfloat16 or int8, got {x_dtype}")
    return int(_abi.load().gptq_packed_linear_workspace_bytes(n, r, d, bits, group,
                                                              _DTYPE[x_dtype], int(permuted)))


def gptq_packed_linear(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                       zeros: torch.Tensor, bits: int, group: int, *,
                       x_scales: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                       perm: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                       y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """y [n, r] = x [n, d] W^^T + bias from the packed layer, for any number of tokens.

    x fp16 or bf16, or int8 codes with ``x_scales`` fp32 [n] (as
    ``gptq_rmsnorm_int8`` returns them).  y has ``dtype`` (or the given y's type):
    x's own type by default (fp16 for int8 x), or float32.  ``perm`` is
    ``gptq_regroup``'s order when the layer was quantised with act-order and x is
    in its own column order.
    """
    lib = _abi.load()
    _activations(x, (torch.float16, torch.bfloat16, torch.int8))
    n, d = x.shape
    r, dev = qweight.shape[0], x.device
    if bits not in (2, 3, 4, 8) or (group != -1 and (group <= 0 or d % group)):
        raise GPTQError(1, "gptq_packed_linear")
    G = 1 if group == -1 else d // group
    if y is None:
        if dtype is None:
            dtype = torch.float16 if x.dtype == torch.int8 else x.dtype
        with _on(stream):
            y = torch.empty((n, r), dtype=dtype, device=dev)
    elif dtype is not None and y.dtype != dtype:
        raise ValueError(f"y must be {dtype}, got {y.dtype}")
    if y.dtype not in _DTYPE:
        raise ValueError(f"y must be float16, bfloat16 or float32, got {y.dtype}")
    xt = _DTYPE[x.dtype]
    if workspace is None and (perm is not None or xt == 3):   # 16-bit x in order needs none
        need = lib.gptq_packed_linear_workspace_bytes(n, r, d, bits, group, xt, perm is not None)
        if need:
            with _on(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None and workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}, got {workspace.device}")
    _check(_launch(
        dev, stream, lib.gptq_packed_linear, _shaped(x, x.dtype, (n, d), dev, "x"), xt,
        _shaped(x_scales, torch.float32, (n,), dev, "x_scales"), n,
        _shaped(qweight, torch.int32, (r, d * bits // 32), dev, "qweight"),
        _shaped(scales, torch.float32, (r, G), dev, "scales"),
        _shaped(zeros, torch.int32, (r, G), dev, "zeros"),
        _shaped(perm, torch.int32, (d,), dev, "perm"), r, d, bits, group,
        _shaped(bias, y.dtype, (r,), dev, "bias"), _shaped(y, y.dtype, (n, r), dev, "y"),
        _DTYPE[y.dtype], _ptr(workspace, None, "workspace"),
        0 if workspace is None else workspace.numel() * workspace.element_size()),
        "gptq_packed_linear")
    return y


def gptq_regroup(qweight: torch.Tensor, g_idx: torch.Tensor, bits: int, group: int, *,
                 out: torch.Tensor | None = None, perm: torch.Tensor | None = None,
                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The columns of a packed act-order layer sorted by group, and their order:
    column j of the first result is column perm[j] of ``qweight``.  Waits until the
    order has been checked; the columns follow on the stream."""
    lib = _abi.load()
    if not g_idx.is_cuda or g_idx.dim() != 1:
        raise ValueError("g_idx must be a CUDA tensor [d]")
    d, r, dev = g_idx.shape[0], qweight.shape[0], g_idx.device
    with _on(stream):
        if out is None:
            out = torch.empty_like(qweight)
        if perm is None:
            perm = torch.empty_like(g_idx)
    words = (r, d * bits // 32)
    _check(_launch(
        dev, stream, lib.gptq_regroup, _shaped(qweight, torch.int32, words, dev, "qweight"),
        _shaped(g_idx, torch.int32, (d,), dev, "g_idx"), r, d, bits, group,
        _shaped(out, torch.int32, words, dev, "out"),
        _shaped(perm, torch.int32, (d,), dev, "perm")), "gptq_regroup")
    return out, perm


_ACTIVATION = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


def _activation(name: str) -> int:
    if name not in _ACTIVATION:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATION)}, got {name!r}")
    return _ACTIVATION[name]


def gptq_int8_weights(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, d: int, bits: int, *,
                      w: torch.Tensor | None = None, w_scales: torch.Tensor | None = None,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """A packed layer with one scale per row (group -1) as 8-bit integers: w int8
    [r, d] = q - zeros, and w_scales fp32 [r], for ``gptq_int8_linear`` and
    ``gptq_int8_gated``.

    Layers of 2, 3 and 4 bits, and 8-bit ones of the symmetric quantiser (``sym=True``); a
    row whose q - zero leaves int8 has scale NaN.
    """
    lib = _abi.load()
    if not qweight.is_cuda or qweight.dim() != 2:
        raise ValueError("qweight must be a CUDA tensor [rows, words]")
    if bits not in (2, 3, 4, 8):
        raise GPTQError(1, "gptq_int8_weights")
    r, dev = qweight.shape[0], qweight.device
    with _on(stream):
        if w is None:
            w = torch.empty((r, d), dtype=torch.int8, device=dev)
        if w_scales is None:
            w_scales = torch.empty(r, dtype=torch.float32, device=dev)
    _check(_launch(
        dev, stream, lib.gptq_int8_weights, _shaped(qweight, torch.int32, (r, d * bits // 32), dev, "qweight"),
        _shaped(scales, torch.float32, (r, 1), dev, "scales"), _shaped(zeros, torch.int32, (r, 1), dev, "zeros"),
        r, d, bits, _shaped(w, torch.int8, (r, d), dev, "w"),
        _shaped(w_scales, torch.float32, (r,), dev, "w_scales")), "gptq_int8_weights")
    return w, w_scales


def _result(y: torch.Tensor | None, dtype: torch.dtype | None, shape: tuple, device: torch.device,
            stream) -> torch.Tensor:
    """The given y, or a new one (fp16 by default)."""
    if y is None:
        with _on(stream):
            y = torch.empty(shape, dtype=torch.float16 if dtype is None else dtype, device=device)
    elif dtype is not None and y.dtype != dtype:
        raise ValueError(f"y must be {dtype}, got {y.dtype}")
    if y.dtype not in (torch.float16, torch.bfloat16, torch.float32):
        raise ValueError(f"y must be float16, bfloat16 or float32, got {y.dtype}")
    return y


def gptq_int8_linear(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, *,
                     bias: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                     y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [n, r] = x_scales w_scales (x w^T) + bias in 8-bit integers, for any number of tokens.

    x int8 [n, d] with x_scales fp32 [n] (from ``gptq_rmsnorm_int8`` or
    ``gptq_activation_int8``), w int8 [r, d] with w_scales fp32 [r] (from
    ``gptq_int8_weights``).  y has ``dtype`` (or the given y's type): fp16 by default,
    bf16 or fp32; a bias has it too.  Sums are exact.
    """
    lib = _abi.load()
    _activations(x, (torch.int8,))
    n, d = x.shape
    r, dev = w.shape[0], x.device
    y = _result(y, dtype, (n, r), dev, stream)
    _check(_launch(
        dev, stream, lib.gptq_int8_linear, _shaped(x, torch.int8, (n, d), dev, "x"),
        _shaped(x_scales, torch.float32, (n,), dev, "x_scales"), n, _shaped(w, torch.int8, (r, d), dev, "w"),
        _shaped(w_scales, torch.float32, (r,), dev, "w_scales"), r, d, _shaped(bias, y.dtype, (r,), dev, "bias"),
        _shaped(y, y.dtype, (n, r), dev, "y"), _DTYPE[y.dtype]), "gptq_int8_linear")
    return y


def gptq_int8_gated(x: torch.Tensor, x_scales: torch.Tensor, gate: torch.Tensor, gate_scales: torch.Tensor,
                    up: torch.Tensor, up_scales: torch.Tensor, *, activation: str = "silu",
                    gate_bias: torch.Tensor | None = None, up_bias: torch.Tensor | None = None,
                    dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """y [n, r] = act(gate product) * (up product), both as ``gptq_int8_linear``, in one
    kernel.  ``activation``: "none", "relu", "silu" or "gelu" (with erf)."""
    lib = _abi.load()
    _activations(x, (torch.int8,))
    act = _activation(activation)
    n, d = x.shape
    r, dev = gate.shape[0], x.device
    y = _result(y, dtype, (n, r), dev, stream)
    _check(_launch(
        dev, stream, lib.gptq_int8_gated, _shaped(x, torch.int8, (n, d), dev, "x"),
        _shaped(x_scales, torch.float32, (n,), dev, "x_scales"), n,
        _shaped(gate, torch.int8, (r, d), dev, "gate"), _shaped(gate_scales, torch.float32, (r,), dev, "gate_scales"),
        _shaped(up, torch.int8, (r, d), dev, "up"), _shaped(up_scales, torch.float32, (r,), dev, "up_scales"), r, d,
        _shaped(gate_bias, y.dtype, (r,), dev, "gate_bias"), _shaped(up_bias, y.dtype, (r,), dev, "up_bias"), act,
        _shaped(y, y.dtype, (n, r), dev, "y"), _DTYPE[y.dtype]), "gptq_int8_gated")
    return y


def gptq_activation_int8(x: torch.Tensor, up: torch.Tensor | None = None, *, activation: str = "silu",
                         perm: torch.Tensor | None = None, xhat: bool = False, outputs: dict | None = None,
                         stream=None) -> dict:
    """u = act(x), times ``up`` when given, in symmetric 8-bit codes with one scale per token.

    x and up [n, d] fp16 or bf16; ``activation`` as ``gptq_int8_gated``.  Returns ``codes``
    int8 [n, d], ``scales`` fp32 [n], and ``xhat`` = scales * codes in x's type when asked
    for; ``perm`` and ``outputs`` as ``gptq_rmsnorm_int8``.
    """
    lib = _abi.load()
    _activations(x, (torch.float16, torch.bfloat16))
    act = _activation(activation)
    n, d = x.shape
    dev, T = x.device, x.dtype
    codes = scales = xh = None
    if outputs:
        codes, scales, xh = outputs.get("codes"), outputs.get("scales"), outputs.get("xhat")
    if codes is None or scales is None or (xhat and xh is None):
        with _on(stream):
            if codes is None:
                codes = torch.empty((n, d), dtype=torch.int8, device=dev)
            if scales is None:
                scales = torch.empty(n, dtype=torch.float32, device=dev)
            if xh is None and xhat:
                xh = torch.empty((n, d), dtype=T, device=dev)
    _check(_launch(
        dev, stream, lib.gptq_activation_int8, _shaped(x, T, (n, d), dev, "x"), _shaped(up, T, (n, d), dev, "up"),
        _DTYPE[T], n, d, act, _shaped(perm, torch.int32, (d,), dev, "perm"),
        _shaped(codes, torch.int8, (n, d), dev, "codes"), _shaped(scales, torch.float32, (n,), dev, "scales"),
        _shaped(xh, T, (n, d), dev, "xhat")), "gptq_activation_int8")
    res = {"codes": codes, "scales": scales}
    if xh is not None:
        res["xhat"] = xh
    return res


def gptq_pack(codes: torch.Tensor, bits: int, qweight: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    lib = _abi.load()
    r, d = codes.shape
    if qweight is None:
        qweight = torch.empty((r, d * bits // 32), dtype=torch.int32, device=codes.device)
    _check(lib.gptq_pack(_ptr(codes, torch.uint8, "codes"), r, d, bits,
                         _ptr(qweight, torch.int32, "qweight"), _stream(stream)), "gptq_pack")
    return qweight


def gptq_layer_host_workspace_bytes(r: int, d: int, n: int, bits: int, group: int,
                                    block: int = 128, act_order: bool = False,
                                    sym: bool = False, static_groups: bool = False) -> int:
    return int(_abi.load().gptq_layer_host_workspace_bytes(
        r, d, n, bits, group, block, _options(act_order, sym, static_groups)))


def gptq_solve_layer_host(X: torch.Tensor, W: torch.Tensor, *, bits: int, group: int,
                          block: int = 128, damp: float = 0.01, act_order: bool = False,
                          sym: bool = False, static_groups: bool = False,
                          dev_workspace: torch.Tensor, outputs: dict, stream=None) -> float:
    """Whole layer from host (CPU, ideally pinned) tensors; fills ``outputs`` host tensors."""
    lib = _abi.load()
    n, d = X.shape
    r = W.shape[0]
    for t, name in ((X, "X"), (W, "W")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    if X.dtype != torch.float16 or W.dtype != torch.float32:
        raise ValueError("X must be float16 and W float32")
    loss = ctypes.c_double(0.0)
    gi = outputs.get("g_idx")
    _check(lib.gptq_solve_layer_host(
        X.data_ptr(), n, W.data_ptr(), r, d, bits, group, block, float(damp),
        _options(act_order, sym, static_groups),
        outputs["qweight"].data_ptr(), outputs["scales"].data_ptr(), outputs["zeros"].data_ptr(),
        gi.data_ptr() if gi is not None else None, ctypes.byref(loss),
        _ptr(dev_workspace, None, "dev_workspace"),
        dev_workspace.numel() * dev_workspace.element_size(), _stream(stream)),
        "gptq_solve_layer_host")
    return loss.value


def gptq_check_device_status(stream=None) -> int:
    return int(_abi.load().gptq_check_device_status(_stream(stream)))


def gptq_launch_count() -> int:
    return int(_abi.load().gptq_launch_count())


def gptq_set_phase_timing(enable: bool) -> None:
    _abi.load().gptq_set_phase_timing(int(enable))


def gptq_last_phase_ms() -> list[float]:
    buf = (ctypes.c_float * 4)()
    n = _abi.load().gptq_last_phase_ms(buf, 4)
    return [float(buf[i]) for i in range(n)]


def gptq_factor_plan(d: int, outer_cols: int = 0, side_streams: bool = True) -> str:
    """The factorisation's launches and stream events for a d x d H_d (no GPU used)."""
    lib = _abi.load()
    n = lib.gptq_factor_plan(d, outer_cols, int(side_streams), None, 0)
    if n == 0:
        raise GPTQError(1, "gptq_factor_plan: invalid arguments")
    buf = ctypes.create_string_buffer(n)
    lib.gptq_factor_plan(d, outer_cols, int(side_streams), buf, n)
    return buf.value.decode()


def gptq_gemm_pair_form() -> tuple[int, str]:
    """(form, probe record) of the two-CTA product on the current device: 0-5 a
    cluster launch form, 6 the one-CTA fallback, -1 not probed yet."""
    lib = _abi.load()
    buf = ctypes.create_string_buffer(512)
    form = lib.gptq_gemm_pair_form(buf, 512)
    return int(form), buf.value.decode()


def gptq_set_gemm_pair(enable: bool) -> bool:
    """Run products with two or more row tiles on CTA pairs (True) or one CTA per
    tile (False, the default); returns the previous setting."""
    return bool(_abi.load().gptq_set_gemm_pair(int(bool(enable))))
