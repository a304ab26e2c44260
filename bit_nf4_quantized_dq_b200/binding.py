"""Thin Python binding over the C ABI in include/qlora_nf4.h.

Argument marshalling only: PyTorch provides device memory and the current stream, every
step of the computation runs in the library's CUDA kernels.  There is no fallback: if the
shared library is missing or cannot be loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

_LIB: Optional[ctypes.CDLL] = None

c_void_p = ctypes.c_void_p
c_int64 = ctypes.c_int64
c_int = ctypes.c_int
c_size_t = ctypes.c_size_t
c_float = ctypes.c_float
c_double = ctypes.c_double

# name -> (restype, argtypes); mirrors include/qlora_nf4.h
SIGNATURES = {
    "qnf4_version": (c_int, []),
    "qnf4_last_error": (ctypes.c_char_p, []),
    "qnf4_device_error": (c_int, [c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "qnf4_selftest_bounded_wait": (c_int, [ctypes.c_uint64, c_void_p]),
    "nf4_quantize_workspace_bytes": (c_size_t, [c_int64]),
    "nf4_quantize_dq": (c_int, [c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_size_t, c_void_p]),
    "nf4_quantize_dq_noalloc": (c_int, [c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "nf4_dequant": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p]),
    "qlora_linear_fwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int]),
    "qlora_linear_fwd": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p,
                                 c_void_p, c_size_t, c_void_p]),
    "qlora_linear_bwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int]),
    "qlora_linear_bwd": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_float,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "nf4_e4m3_encode": (c_int, [c_void_p, c_int64, c_void_p, c_int, c_void_p]),
    "qnf4_quantize_workspace_bytes_ex": (c_size_t, [c_int64, c_int]),
    "qnf4_quantize_ex": (c_int, [c_void_p, c_int64, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_size_t, c_void_p]),
    "qnf4_dequant_ex": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p]),
    "qlora_linear_fwd_ex": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_int, c_int, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p,
                                    c_void_p, c_size_t, c_void_p]),
    "qnf4_paged_alloc": (c_int, [c_size_t, ctypes.POINTER(c_void_p)]),
    "qnf4_paged_free": (c_int, [c_void_p]),
    "qnf4_paged_prefetch": (c_int, [c_void_p, c_size_t, c_int, c_void_p]),
    "qlora_adamw_step": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_double, c_double,
                                 c_double, c_double, c_double, c_int, c_void_p]),
    "qlora_merge_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int, c_int]),
    "qlora_merge_requantize": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int, c_int,
                                       c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_size_t, c_void_p]),
    "qlora_linear_bwd_ex": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64, c_int, c_int,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_float,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "qnf4_act8_quantize": (c_int, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p]),
    "qnf4_act8_dequant": (c_int, [c_void_p, c_void_p, c_int64, c_int64, c_void_p, c_void_p]),
    "qlora_linear_bwd_act8": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int64, c_int, c_int,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_float,
                                      c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "qlora_rmsnorm_fwd": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_double, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p]),
    "qlora_rmsnorm_bwd_workspace_bytes": (c_size_t, [c_int64, c_int64]),
    "qlora_rmsnorm_bwd": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_void_p,
                                  c_void_p, c_void_p, c_size_t, c_void_p]),
    "qlora_linear_epi_fwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int]),
    "qlora_linear_epi_fwd": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p, c_int, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "qlora_epilogue_bwd_workspace_bytes": (c_size_t, [c_int64, c_int64]),
    "qlora_epilogue_bwd": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int, c_void_p, c_void_p,
                                   c_void_p, c_size_t, c_void_p]),
    "qnf4_set_timing_events": (c_int, [c_void_p, c_int]),
    "qlora_linear_plan": (c_int, [c_int64, c_int64, c_int64, c_int, ctypes.POINTER(c_int),
                                  ctypes.POINTER(c_int), ctypes.POINTER(c_int), ctypes.POINTER(c_int)]),
}


class QNF4Error(RuntimeError):
    pass


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library (building it first if it is missing or stale and nvcc exists)."""
    global _LIB
    if _LIB is None:
        path = _build.LIB_PATH
        if not os.path.exists(path) or _build.is_stale():
            try:
                _build.build()
            except Exception as e:  # no nvcc: only an existing library can be used
                if not os.path.exists(path):
                    raise QNF4Error(f"the CUDA library {path} is missing and cannot be built: {e}")
        handle = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def _check(rc: int, what: str) -> None:
    if rc != 0:
        msg = lib().qnf4_last_error().decode(errors="replace")
        raise QNF4Error(f"{what} failed with status {rc}: {msg}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise QNF4Error("operands must be contiguous CUDA tensors")


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _bf16_bits(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.bfloat16:
        raise QNF4Error("expected a bfloat16 tensor")
    return t


def check_device_error() -> int:
    """Synchronise the current stream; raise if a kernel gave up waiting."""
    word = ctypes.c_uint32(0)
    rc = lib().qnf4_device_error(_stream(), ctypes.byref(word))
    if rc != 0:
        raise QNF4Error(f"device error word 0x{word.value:x}: {lib().qnf4_last_error().decode()}")
    return word.value


CODEBOOKS = {"nf4": 0, "fp4_e2m1": 1, "int4": 2}   # QNF4_CODEBOOK_* in include/qlora_nf4.h


class NF4Tensor:
    """A quantized weight: 4-bit codes and their block scales.

    With double quantization (the default): E4M3 scale codes, fp32 group constants `c2` and
    the fp32 mean.  Without it: `c2` holds one fp32 absmax per block and `scale_codes` and
    `mean` are None.  `codebook` names the 16 levels ("nf4", "fp4_e2m1" or "int4")."""

    def __init__(self, codes, scale_codes, c2, mean, shape, codebook: str = "nf4", double_quant: bool = True):
        if codebook not in CODEBOOKS:
            raise QNF4Error(f"unknown code book {codebook!r}")
        self.codes = codes
        self.scale_codes = scale_codes
        self.c2 = c2
        self.mean = mean
        self.shape = tuple(shape)
        self.codebook = codebook
        self.double_quant = bool(double_quant)

    @property
    def scales(self):
        return self.c2

    def _format(self):
        return CODEBOOKS[self.codebook], 1 if self.double_quant else 0

    @property
    def numel(self) -> int:
        n = 1
        for d in self.shape:
            n *= d
        return n

    def nbytes(self) -> int:
        n = self.codes.numel() + 4 * self.c2.numel()
        if self.double_quant:
            n += self.scale_codes.numel() + 4 * self.mean.numel()
        return n


class Act8Tensor:
    """An 8-bit checkpoint of a bf16 tensor [M][K]: E4M3 codes [M][ld] (ld = K rounded up to 16)
    and scale bytes [M][ceil(K / 32)], one power of two per row and 32 features: E4M3(code) * 2^(byte - 127),
    NaN for the codes 0x7F and 0xFF and for the byte 255."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, shape):
        self.codes = codes
        self.scales = scales
        self.shape = tuple(shape)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _require_act8(a: "Act8Tensor", device, what: str) -> None:
    if not isinstance(a, Act8Tensor) or len(a.shape) != 2:
        raise QNF4Error(f"{what} must be the 8-bit checkpoint of a matrix")
    M, K = a.shape
    for t, cols, name in ((a.codes, (K + 15) // 16 * 16, "codes"), (a.scales, (K + 31) // 32, "scales")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or tuple(t.shape) != (M, cols) \
                or not t.is_contiguous() or t.device != device:
            raise QNF4Error(f"the {name} of {what} must be a contiguous uint8 tensor [{M}][{cols}] on {device}")


def quantize(W: torch.Tensor, codebook: str = "nf4", double_quant: bool = True,
             workspace: Optional[torch.Tensor] = None) -> NF4Tensor:
    """Blockwise 4-bit quantization of a bf16 weight with any of the code books, with or
    without double quantization of the block scales."""
    if codebook == "nf4" and double_quant:
        return nf4_quantize_dq(W, workspace)
    W = _bf16_bits(W)
    _require_cuda(W)
    numel = W.numel()
    nb = (numel + 63) // 64
    ng = (nb + 255) // 256
    dev = W.device
    codes = torch.empty(32 * nb, dtype=torch.uint8, device=dev)
    if double_quant:
        sc = torch.empty(nb, dtype=torch.uint8, device=dev)
        scales = torch.empty(ng, dtype=torch.float32, device=dev)
        mean = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        sc, mean = None, None
        scales = torch.empty(nb, dtype=torch.float32, device=dev)
    out = NF4Tensor(codes, sc, scales, mean, W.shape, codebook, double_quant)
    cb, dq = out._format()
    L = lib()
    need = L.qnf4_quantize_workspace_bytes_ex(numel, dq)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, dev)
    _check(L.qnf4_quantize_ex(_ptr(W), numel, cb, dq, _ptr(codes), _ptr(sc), _ptr(scales), _ptr(mean),
                              _ptr(workspace), workspace.numel(), _stream()), "qnf4_quantize_ex")
    return out


def nf4_quantize_dq(W: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> NF4Tensor:
    """Quantize a bf16 weight (any shape, flattened row-major) to NF4 + DQ."""
    W = _bf16_bits(W)
    _require_cuda(W)
    numel = W.numel()
    nb = (numel + 63) // 64
    ng = (nb + 255) // 256
    dev = W.device
    codes = torch.empty(32 * nb, dtype=torch.uint8, device=dev)
    scale_codes = torch.empty(nb, dtype=torch.uint8, device=dev)
    c2 = torch.empty(ng, dtype=torch.float32, device=dev)
    mean = torch.empty(1, dtype=torch.float32, device=dev)
    L = lib()
    need = L.nf4_quantize_workspace_bytes(numel)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, dev)
    _check(L.nf4_quantize_dq(_ptr(W), numel, _ptr(codes), _ptr(scale_codes), _ptr(c2), _ptr(mean),
                             _ptr(workspace), workspace.numel(), _stream()), "nf4_quantize_dq")
    return NF4Tensor(codes, scale_codes, c2, mean, W.shape)


def _check_out_buffer(t: torch.Tensor, dtype, count: int, device, name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise QNF4Error(f"out.{name} must be a contiguous {dtype} tensor on {device}")
    if t.numel() < count:
        raise QNF4Error(f"out.{name} holds {t.numel()} elements, the weight needs {count}")


def nf4_quantize_dq_noalloc(W: torch.Tensor, out: Optional[NF4Tensor] = None) -> NF4Tensor:
    """nf4_quantize_dq without a workspace: the library's static scratch holds the absmax and
    group sums (numel <= NOALLOC_MAX_NUMEL; overlapping calls on one device race on it).  Pass
    `out` to write into existing buffers, so that the call itself allocates nothing; they are
    checked against W (device, dtype, contiguity, size) before the call."""
    W = _bf16_bits(W)
    _require_cuda(W)
    numel = W.numel()
    nb = (numel + 63) // 64
    ng = (nb + 255) // 256
    dev = W.device
    if out is None:
        out = NF4Tensor(torch.empty(32 * nb, dtype=torch.uint8, device=dev),
                        torch.empty(nb, dtype=torch.uint8, device=dev),
                        torch.empty(ng, dtype=torch.float32, device=dev),
                        torch.empty(1, dtype=torch.float32, device=dev), W.shape)
    else:
        _check_out_buffer(out.codes, torch.uint8, 32 * nb, dev, "codes")
        _check_out_buffer(out.scale_codes, torch.uint8, nb, dev, "scale_codes")
        _check_out_buffer(out.c2, torch.float32, ng, dev, "c2")
        _check_out_buffer(out.mean, torch.float32, 1, dev, "mean")
    with torch.cuda.device(dev):
        _check(lib().nf4_quantize_dq_noalloc(_ptr(W), numel, _ptr(out.codes), _ptr(out.scale_codes), _ptr(out.c2),
                                             _ptr(out.mean), _stream()), "nf4_quantize_dq_noalloc")
    out.shape = tuple(W.shape)
    return out


NOALLOC_MAX_NUMEL = 1 << 28   # QNF4_NOALLOC_MAX_NUMEL


def nf4_dequant(q: NF4Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """NF4 + DQ -> bf16 tensor of the original shape."""
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.codes.device)
    _require_cuda(out, q.codes)
    cb, dq = q._format()
    _check(lib().qnf4_dequant_ex(_ptr(q.codes), cb, dq, _ptr(q.scale_codes), _ptr(q.c2), _ptr(q.mean), q.numel,
                                 _ptr(out), _stream()), "qnf4_dequant_ex")
    return out


def qlora_linear_fwd(x: torch.Tensor, q: NF4Tensor, A: torch.Tensor, B: torch.Tensor, s: float,
                     workspace: Optional[torch.Tensor] = None):
    """y = x W'^T + s (x A^T) B^T.  Returns (y, t_saved).

    This call takes every token count through the same tiles.  For up to 16 tokens qlora_linear_epilogue_fwd(x, q,
    A, B, s, save=True) gives the same y and t, up to the order of their sums, in 0.4 to 0.8 of the time."""
    _require_cuda(x, A, B)
    M, K = x.shape
    N = q.shape[0]
    r = A.shape[0]
    if q.shape != (N, K) or tuple(A.shape) != (r, K) or tuple(B.shape) != (N, r):
        raise QNF4Error("shape mismatch between x, W, A and B")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    t = torch.empty((M, r), dtype=torch.float32, device=x.device)
    L = lib()
    need = L.qlora_linear_fwd_workspace_bytes(M, K, N, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, x.device)
    cb, dq = q._format()
    _check(L.qlora_linear_fwd_ex(_ptr(x), M, K, N, cb, dq, _ptr(q.codes), _ptr(q.scale_codes), _ptr(q.c2),
                                 _ptr(q.mean), _ptr(A), _ptr(B), r, float(s), _ptr(y), _ptr(t), _ptr(workspace),
                                 workspace.numel(), _stream()), "qlora_linear_fwd")
    return y, t


def qlora_linear_bwd(dY: torch.Tensor, x, t_saved: torch.Tensor, q: NF4Tensor,
                     A: torch.Tensor, B: torch.Tensor, s: float, need_dx: bool = True,
                     workspace: Optional[torch.Tensor] = None):
    """Returns (dX or None, dA, dB).  x is the forward's bf16 input, or an Act8Tensor of it: dX is then the same, dA
    and dB those of the decoded values, up to the order in which the sums of the splits of the tokens are joined."""
    if isinstance(x, Act8Tensor):
        return _linear_bwd_act8(dY, x, t_saved, q, A, B, s, need_dx, workspace)
    _require_cuda(dY, x, t_saved, A, B)
    M, K = x.shape
    N = q.shape[0]
    r = A.shape[0]
    dX = torch.empty((M, K), dtype=torch.bfloat16, device=x.device) if need_dx else None
    dA = torch.empty((r, K), dtype=torch.bfloat16, device=x.device)
    dB = torch.empty((N, r), dtype=torch.bfloat16, device=x.device)
    L = lib()
    need = L.qlora_linear_bwd_workspace_bytes(M, K, N, r)
    if workspace is None or workspace.numel() < need:
        workspace = _ws(need, x.device)
    cb, dq = q._format()
    _check(L.qlora_linear_bwd_ex(_ptr(dY), _ptr(x), _ptr(t_saved), M, K, N, cb, dq, _ptr(q.codes),
                                 _ptr(q.scale_codes), _ptr(q.c2), _ptr(q.mean), _ptr(A), _ptr(B), r, float(s),
                                 _ptr(dX), _ptr(dA), _ptr(dB), _ptr(workspace), workspace.numel(), _stream()),
           "qlora_linear_bwd")
    return dX, dA, dB


def _require(t, dtype, shape, device, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise QNF4Error(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype != dtype or tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise QNF4Error(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}, "
                        f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _require_weight(q: NF4Tensor, device) -> None:
    """The stored parts of a quantized weight: types, sizes and device, as the kernels index them."""
    if not isinstance(q, NF4Tensor) or len(q.shape) != 2:
        raise QNF4Error("the quantized weight must be an NF4Tensor of two dimensions")
    nb = (q.numel + 63) // 64
    _require_part(q.codes, torch.uint8, 32 * nb, device, "codes")
    if q.double_quant:
        _require_part(q.scale_codes, torch.uint8, nb, device, "scale_codes")
        _require_part(q.c2, torch.float32, (nb + 255) // 256, device, "c2")
        _require_part(q.mean, torch.float32, 1, device, "mean")
    else:
        _require_part(q.c2, torch.float32, nb, device, "scales")


def _require_part(t, dtype, count: int, device, name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() < count or t.device != device or not t.is_contiguous():
        raise QNF4Error(f"the weight's {name} must hold {count} contiguous {dtype} elements on {device}")


def _rank(A) -> int:
    """Rows of the adapter A, whose other properties _require checks."""
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise QNF4Error("A must be a matrix")
    return A.shape[0]


def _empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A contiguous matrix (torch.empty takes 2.3 us of a call's 12 to 20 for the same)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _require_gpu(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise QNF4Error(f"{name} must be a CUDA tensor")
    return t.device


def _workspace(given: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    """The caller's workspace where it is large enough, else a new one."""
    if given is None or given.numel() * given.element_size() < need:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if given.device != device or not given.is_contiguous():
        raise QNF4Error(f"the workspace must be a contiguous tensor on {device}")
    return given


def _stream_of(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The same as an integer without building a Stream object (2 us of a call's 14), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(device, what: str, fn, *args) -> None:
    """fn(*args, stream) with `device` current, on that device's current stream."""
    if device.index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(device.index) if _raw_stream else _stream_of(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream_of(device))
    if rc != 0:
        _check(rc, what)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _linear_bwd_act8(dY, x: Act8Tensor, t_saved, q: NF4Tensor, A, B, s: float, need_dx: bool, workspace):
    bf16 = torch.bfloat16
    dev = _require_gpu(dY, "dY")
    _require_act8(x, dev, "x")
    M, K = x.shape
    _require_weight(q, dev)
    N, r = q.shape[0], _rank(A)
    if q.shape[1] != K:
        raise QNF4Error("shape mismatch between x and W")
    _require(dY, bf16, (M, N), dev, "dY")
    _require(t_saved, torch.float32, (M, r), dev, "t_saved")
    _require(A, bf16, (r, K), dev, "A")
    _require(B, bf16, (N, r), dev, "B")
    dX = _empty(M, K, bf16, dev) if need_dx else None
    dA, dB = _empty(r, K, bf16, dev), _empty(N, r, bf16, dev)
    L = lib()
    ws = _workspace(workspace, L.qlora_linear_bwd_workspace_bytes(M, K, N, r), dev)
    cb, dq = q._format()
    _launch(dev, "qlora_linear_bwd_act8", L.qlora_linear_bwd_act8, dY.data_ptr(), x.codes.data_ptr(),
            x.scales.data_ptr(), t_saved.data_ptr(), M, K, N, cb, dq, q.codes.data_ptr(), _addr(q.scale_codes),
            q.c2.data_ptr(), _addr(q.mean), A.data_ptr(), B.data_ptr(), r, float(s), _addr(dX), dA.data_ptr(),
            dB.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return dX, dA, dB


def merge_requantize(q: NF4Tensor, A: torch.Tensor, B: torch.Tensor, s: float, return_merged: bool = False):
    """Fold the adapters into the base and quantize the result again in the same format:
    W'' = bf16(W' + s B A), then quantized.  Returns the new NF4Tensor (and W'' as a bf16
    tensor when `return_merged`)."""
    _require_cuda(A, B, q.codes)
    N, K = q.shape
    r = A.shape[0]
    if tuple(A.shape) != (r, K) or tuple(B.shape) != (N, r):
        raise QNF4Error("shape mismatch between W, A and B")
    dev = q.codes.device
    nb = (N * K + 63) // 64
    ng = (nb + 255) // 256
    codes = torch.empty(32 * nb, dtype=torch.uint8, device=dev)
    if q.double_quant:
        sc = torch.empty(nb, dtype=torch.uint8, device=dev)
        scales = torch.empty(ng, dtype=torch.float32, device=dev)
        mean = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        sc, mean = None, None
        scales = torch.empty(nb, dtype=torch.float32, device=dev)
    out = NF4Tensor(codes, sc, scales, mean, (N, K), q.codebook, q.double_quant)
    merged = torch.empty((N, K), dtype=torch.bfloat16, device=dev) if return_merged else None
    cb, dq = q._format()
    L = lib()
    ws = _ws(L.qlora_merge_workspace_bytes(N, K, dq, 1 if merged is not None else 0), dev)
    _check(L.qlora_merge_requantize(_ptr(q.codes), _ptr(q.scale_codes), _ptr(q.c2), _ptr(q.mean), N, K, cb, dq,
                                    _ptr(A), _ptr(B), r, float(s), _ptr(codes), _ptr(sc), _ptr(scales), _ptr(mean),
                                    _ptr(merged), _ptr(ws), ws.numel(), _stream()), "qlora_merge_requantize")
    return (out, merged) if return_merged else out


def set_timing_events(events) -> None:
    """Record these torch.cuda.Event objects at the stage boundaries of later fwd / bwd calls
    made from this thread (see qnf4_set_timing_events); None stops recording."""
    global _EVENT_ARRAY
    if not events:
        _EVENT_ARRAY = None
        _check(lib().qnf4_set_timing_events(None, 0), "qnf4_set_timing_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _EVENT_ARRAY = arr                       # keep the handle array alive while recording
    _check(lib().qnf4_set_timing_events(ctypes.cast(arr, ctypes.c_void_p), len(events)),
           "qnf4_set_timing_events")


_EVENT_ARRAY = None


def linear_plan(M: int, K: int, N: int, r: int) -> dict:
    """Kernel launches per forward / backward call and the fused GEMMs' K-split factors."""
    v = [c_int(0) for _ in range(4)]
    _check(lib().qlora_linear_plan(M, K, N, r, *[ctypes.byref(x) for x in v]), "qlora_linear_plan")
    return {"fwd_launches": v[0].value, "bwd_launches": v[1].value, "fwd_splits": v[2].value,
            "dx_splits": v[3].value}


def e4m3_encode(v: torch.Tensor, mode: int = 0) -> torch.Tensor:
    _require_cuda(v)
    out = torch.empty(v.numel(), dtype=torch.uint8, device=v.device)
    _check(lib().nf4_e4m3_encode(_ptr(v), v.numel(), _ptr(out), mode, _stream()), "nf4_e4m3_encode")
    return out
