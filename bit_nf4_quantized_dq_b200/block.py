"""The operators around the QLoRA linear in a decoder block: the norm in front of it, its bias,
activation and residual, and the 8-bit checkpoints that its backward pass reads.

Argument marshalling only, as in binding.py: every call checks its operands' types, shapes,
layout and device, allocates its outputs, and runs the library's kernels on the current stream
of the operands' device.  A training step of one sublayer:

    y, h, rstd, y8 = rmsnorm_fwd(x, w, residual=res, act8=True)     # y8 is kept, y is not
    g, t, z = qlora_linear_epilogue_fwd(y, W, A, B, s, activation="silu", save=True)
    ...
    dZ, _ = epilogue_bwd(dG, z, "silu")
    dY, dA, dB = qlora_linear_bwd(dZ, y8, t, W, A, B, s)
    dx, dw = rmsnorm_bwd(dY, h, rstd, w, dh=dH)
"""

from __future__ import annotations

from typing import Optional, Union

import torch

from .binding import (
    Act8Tensor, NF4Tensor, QNF4Error, _addr, _empty, _launch, _rank, _require, _require_act8, _require_gpu, _require_weight,
    _workspace, lib,
)

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # QNF4_ACT_*


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise QNF4Error(f"unknown activation {name!r}")
    return ACTIVATIONS[name]


def _matrix(t, name: str):
    """(device, rows, columns) of a contiguous bf16 matrix."""
    dev = _require_gpu(t, name)
    if t.dim() != 2 or t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise QNF4Error(f"{name} must be a contiguous bfloat16 matrix, got {t.dtype} {tuple(t.shape)}")
    return dev, t.shape[0], t.shape[1]


def _empty_act8(M: int, K: int, dev) -> Act8Tensor:
    return Act8Tensor(_empty(M, (K + 15) // 16 * 16, torch.uint8, dev), _empty(M, (K + 31) // 32, torch.uint8, dev), (M, K))


def act8_quantize(x: torch.Tensor) -> Act8Tensor:
    """8-bit checkpoint of a bf16 matrix (E4M3 codes, a power-of-two scale per row and 32 columns)."""
    dev, M, K = _matrix(x, "x")
    out = _empty_act8(M, K, dev)
    _launch(dev, "qnf4_act8_quantize", lib().qnf4_act8_quantize, x.data_ptr(), M, K, out.codes.data_ptr(),
            out.scales.data_ptr())
    return out


def act8_dequant(a: Act8Tensor) -> torch.Tensor:
    """The values of an 8-bit checkpoint, as bf16 (exact)."""
    dev = _require_gpu(getattr(a, "codes", None), "a.codes")
    _require_act8(a, dev, "a")
    M, K = a.shape
    out = _empty(M, K, torch.bfloat16, dev)
    _launch(dev, "qnf4_act8_dequant", lib().qnf4_act8_dequant, a.codes.data_ptr(), a.scales.data_ptr(), M, K,
            out.data_ptr())
    return out


def rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None,
                act8: bool = False):
    """Root-mean-square norm of x + residual.  Returns (y, h, rstd, y8): the normed output, the sum
    as bf16 (x itself without a residual), the fp32 reciprocal roots, and with ``act8`` the 8-bit
    checkpoint of y (else None).  h and rstd are what rmsnorm_bwd reads."""
    dev, M, K = _matrix(x, "x")
    _require(weight, torch.bfloat16, (K,), dev, "weight")
    if residual is not None:
        _require(residual, torch.bfloat16, (M, K), dev, "residual")
    y = torch.empty_like(x)
    h = torch.empty_like(x) if residual is not None else None
    rstd = torch.empty(M, dtype=torch.float32, device=dev)
    y8 = _empty_act8(M, K, dev) if act8 else None
    _launch(dev, "qlora_rmsnorm_fwd", lib().qlora_rmsnorm_fwd, x.data_ptr(), _addr(residual), weight.data_ptr(), M, K,
            float(eps), y.data_ptr(), _addr(h), rstd.data_ptr(), y8.codes.data_ptr() if act8 else None,
            y8.scales.data_ptr() if act8 else None)
    return y, (x if h is None else h), rstd, y8


def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                dh: Optional[torch.Tensor] = None, need_dweight: bool = False):
    """Gradients of rmsnorm_fwd: (dx, dweight or None).  dx is the gradient of x and of the
    residual alike; ``dh`` is the gradient that reaches h through the residual stream."""
    dev, M, K = _matrix(dy, "dy")
    _require(h, torch.bfloat16, (M, K), dev, "h")
    _require(rstd, torch.float32, (M,), dev, "rstd")
    _require(weight, torch.bfloat16, (K,), dev, "weight")
    if dh is not None:
        _require(dh, torch.bfloat16, (M, K), dev, "dh")
    dx = torch.empty_like(dy)
    L = lib()
    dw = ws = None
    if need_dweight:
        dw = torch.empty(K, dtype=torch.bfloat16, device=dev)
        ws = _workspace(None, L.qlora_rmsnorm_bwd_workspace_bytes(M, K), dev)
    _launch(dev, "qlora_rmsnorm_bwd", L.qlora_rmsnorm_bwd, dy.data_ptr(), _addr(dh), h.data_ptr(), weight.data_ptr(),
            rstd.data_ptr(), M, K, dx.data_ptr(), _addr(dw), _addr(ws), 0 if ws is None else ws.numel())
    return dx, dw


def qlora_linear_epilogue_fwd(x: torch.Tensor, q: NF4Tensor, A: Optional[torch.Tensor], B: Optional[torch.Tensor],
                              s: float, bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                              residual: Optional[torch.Tensor] = None, save: bool = False,
                              workspace: Optional[torch.Tensor] = None):
    """y = act(x W'^T + s (x A^T) B^T + bias) + residual.  Returns (y, t, z).

    ``activation``: None, "relu", "silu", "gelu" or "gelu_tanh".  A and B may both be None (a base
    without adapters, or with merged ones).  With ``save`` the call also keeps what the backward
    pass reads: t (None without adapters) and the pre-activation z in bf16 (None without an
    activation); without it both are None."""
    act = _activation(activation)
    bf16 = torch.bfloat16
    dev, M, K = _matrix(x, "x")
    _require_weight(q, dev)
    N = q.shape[0]
    if q.shape[1] != K:
        raise QNF4Error("shape mismatch between x and W")
    if (A is None) != (B is None):
        raise QNF4Error("give both adapters or neither")
    r = 0
    if A is not None:
        r = _rank(A)
        _require(A, bf16, (r, K), dev, "A")
        _require(B, bf16, (N, r), dev, "B")
    if bias is not None:
        _require(bias, bf16, (N,), dev, "bias")
    if residual is not None:
        _require(residual, bf16, (M, N), dev, "residual")
    y = _empty(M, N, bf16, dev)
    t = _empty(M, r, torch.float32, dev) if save and r else None
    z = _empty(M, N, bf16, dev) if save and act else None
    L = lib()
    ws = _workspace(workspace, L.qlora_linear_epi_fwd_workspace_bytes(M, K, N, r), dev)
    cb, dq = q._format()
    _launch(dev, "qlora_linear_epi_fwd", L.qlora_linear_epi_fwd, x.data_ptr(), M, K, N, cb, dq, q.codes.data_ptr(),
            _addr(q.scale_codes), q.c2.data_ptr(), _addr(q.mean), _addr(A), _addr(B), r, float(s), _addr(bias), act,
            _addr(residual), y.data_ptr(), _addr(t), _addr(z), ws.data_ptr(), ws.numel() * ws.element_size())
    return y, t, z


def epilogue_bwd(dY: torch.Tensor, z: Union[torch.Tensor, Act8Tensor, None], activation: Optional[str],
                 need_dbias: bool = False):
    """Gradient of the epilogue: (dZ, dbias or None).  dZ = dY * act'(z) goes to qlora_linear_bwd for
    its dY; z is the saved pre-activation or its 8-bit checkpoint.  Without an activation dZ is dY
    itself and z is not read."""
    act = _activation(activation)
    dev, M, N = _matrix(dY, "dY")
    z8 = isinstance(z, Act8Tensor)
    if not act:
        z, z8 = None, False
    elif z8:
        if z.shape != (M, N):
            raise QNF4Error(f"z must have the shape of dY, {(M, N)}, got {z.shape}")
        _require_act8(z, dev, "z")
    elif z is None:
        raise QNF4Error("the activation's gradient needs z")
    else:
        _require(z, torch.bfloat16, (M, N), dev, "z")
    if not act and not need_dbias:
        return dY, None
    dZ = torch.empty_like(dY) if act else None
    L = lib()
    db = ws = None
    if need_dbias:
        db = torch.empty(N, dtype=torch.bfloat16, device=dev)
        ws = _workspace(None, L.qlora_epilogue_bwd_workspace_bytes(M, N), dev)
    _launch(dev, "qlora_epilogue_bwd", L.qlora_epilogue_bwd, dY.data_ptr(), None if z8 else _addr(z),
            z.codes.data_ptr() if z8 else None, z.scales.data_ptr() if z8 else None, M, N, act, _addr(dZ), _addr(db),
            _addr(ws), 0 if ws is None else ws.numel())
    return (dY if dZ is None else dZ), db
