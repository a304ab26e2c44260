"""Refusals of the operators around the linear, on the host before any device work: the C ABI with
addresses that are never dereferenced, and the binding's checks of its operands."""

import ctypes

import pytest
import torch

import bit_nf4_quantized_dq_b200 as q
from bit_nf4_quantized_dq_b200 import binding

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40


def test_act8_refusals():
    L = binding.lib()
    assert L.qnf4_act8_quantize(None, 4, 64, FAKE, FAKE, None) == -1
    assert L.qnf4_act8_quantize(FAKE, 0, 64, FAKE, FAKE, None) == -1
    assert L.qnf4_act8_quantize(FAKE, 4, -8, FAKE, FAKE, None) == -1
    assert L.qnf4_act8_quantize(FAKE, 4, 60, FAKE, FAKE, None) == -2
    assert L.qnf4_act8_quantize(FAKE, 1 << 31, 64, FAKE, FAKE, None) == -1
    assert L.qnf4_act8_quantize(ODD, 4, 64, FAKE, FAKE, None) == -2
    assert L.qnf4_act8_dequant(ODD, FAKE, 4, 64, FAKE, None) == -2
    assert L.qnf4_act8_dequant(FAKE, None, 4, 64, FAKE, None) == -1


def _norm(L, M=4, K=64, eps=1e-5, x=FAKE, res=None, h=None, c=None, s=None):
    return L.qlora_rmsnorm_fwd(x, res, FAKE, M, K, eps, FAKE, h, FAKE, c, s, None)


def test_rmsnorm_refusals():
    L = binding.lib()
    assert _norm(L, M=0) == -1 and _norm(L, K=0) == -1 and _norm(L, K=12) == -2
    assert _norm(L, eps=-1.0) == -1 and _norm(L, eps=float("nan")) == -1 and _norm(L, eps=float("inf")) == -1
    assert _norm(L, x=None) == -1 and _norm(L, x=ODD) == -2
    assert _norm(L, res=FAKE) == -1 and _norm(L, h=FAKE) == -1          # residual and h go together
    assert _norm(L, c=FAKE) == -1 and _norm(L, s=FAKE) == -1            # codes and scales too
    need = L.qlora_rmsnorm_bwd_workspace_bytes(4, 64)
    assert need > 0 and L.qlora_rmsnorm_bwd_workspace_bytes(0, 64) == 0
    bwd = lambda **k: L.qlora_rmsnorm_bwd(FAKE, None, k.get("h", FAKE), FAKE, FAKE, 4, k.get("K", 64), FAKE,  # noqa: E731
                                          k.get("dw"), k.get("ws"), k.get("n", 0), None)
    assert bwd(h=None) == -1 and bwd(K=20) == -2 and bwd(h=ODD) == -2
    assert bwd(dw=FAKE) == -1                                           # dweight needs the workspace
    assert bwd(dw=FAKE, ws=FAKE, n=need - 1) == -6
    assert bwd(dw=FAKE, ws=ODD, n=need) == -2


def _epi(L, M=16, K=64, N=64, r=8, A=FAKE, B=FAKE, act=0, bias=None, res=None, t=None, z=None, ws=FAKE, n=BIG, cb=0):
    return L.qlora_linear_epi_fwd(FAKE, M, K, N, cb, 1, FAKE, FAKE, FAKE, FAKE, A, B, r, 1.0, bias, act, res, FAKE, t, z,
                                  ws, n, None)


def test_linear_epilogue_refusals():
    L = binding.lib()
    assert _epi(L, M=0) == -1 and _epi(L, K=60) == -2 and _epi(L, N=60) == -2
    assert _epi(L, r=12) == -2 and _epi(L, r=264) == -2 and _epi(L, r=0) == -1
    assert _epi(L, A=None) == -1 and _epi(L, B=None) == -1
    assert _epi(L, A=None, B=None) == -1                                # r must be 0 then
    assert _epi(L, A=None, B=None, r=0, t=FAKE) == -1
    assert _epi(L, act=5) == -1 and _epi(L, act=-1) == -1 and _epi(L, cb=3) == -1
    assert _epi(L, bias=ODD) == -2 and _epi(L, res=ODD) == -2 and _epi(L, z=ODD) == -2
    assert _epi(L, ws=None) == -1 and _epi(L, ws=ODD) == -2 and _epi(L, n=16) == -6
    assert L.qlora_linear_epi_fwd_workspace_bytes(16, 64, 64, 0) > 0
    assert L.qlora_linear_epi_fwd_workspace_bytes(16, 64, 64, -1) == 0


def _epi_bwd(L, z=FAKE, zc=None, zs=None, act=2, dz=FAKE, db=None, ws=None, n=0, N=64, dy=FAKE):
    return L.qlora_epilogue_bwd(dy, z, zc, zs, 4, N, act, dz, db, ws, n, None)


def test_epilogue_bwd_refusals():
    L = binding.lib()
    assert _epi_bwd(L, dy=None) == -1 and _epi_bwd(L, dz=None) == -1 and _epi_bwd(L, z=None) == -1
    assert _epi_bwd(L, act=9) == -1 and _epi_bwd(L, N=12) == -2 and _epi_bwd(L, z=ODD) == -2
    assert _epi_bwd(L, z=None, zc=FAKE) == -1 and _epi_bwd(L, z=FAKE, zc=FAKE, zs=FAKE) == -1
    assert _epi_bwd(L, act=0, z=None, dz=None) == -1                    # nothing to compute
    assert _epi_bwd(L, act=0, z=FAKE, dz=None, db=FAKE) == -1
    assert _epi_bwd(L, db=FAKE) == -1
    need = L.qlora_epilogue_bwd_workspace_bytes(4, 64)
    assert _epi_bwd(L, db=FAKE, ws=FAKE, n=need - 1) == -6


def test_linear_bwd_act8_refusals():
    L = binding.lib()
    f = lambda xs=FAKE, xc=FAKE, K=64: L.qlora_linear_bwd_act8(  # noqa: E731
        FAKE, xc, xs, FAKE, 16, K, 64, 0, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 1.0, FAKE, FAKE, FAKE, FAKE, BIG, None)
    assert f(xs=None) == -1 and f(xc=None) == -1 and f(xc=ODD) == -2 and f(K=60) == -2


def test_binding_refuses_cpu_and_wrong_operands():
    bf = torch.bfloat16
    x, w = torch.zeros((4, 64), dtype=bf), torch.zeros(64, dtype=bf)
    for call in (lambda: q.act8_quantize(x), lambda: q.rmsnorm_fwd(x, w),
                 lambda: q.rmsnorm_bwd(x, x, torch.zeros(4), w), lambda: q.epilogue_bwd(x, x, "silu"),
                 lambda: q.act8_dequant(q.Act8Tensor(torch.zeros((4, 64), dtype=torch.uint8),
                                                     torch.zeros((4, 2), dtype=torch.uint8), (4, 64))),
                 lambda: q.epilogue_bwd(x, x, "tanh"),
                 lambda: q.qlora_linear_epilogue_fwd(x, None, None, None, 1.0)):
        with pytest.raises(q.QNF4Error):
            call()


def test_binding_refuses_operands_that_are_missing():
    """The checks behind the calls, on CPU tensors: what is no tensor, no checkpoint, no quantized weight."""
    cpu, bf, u8 = torch.device("cpu"), torch.bfloat16, torch.uint8
    codes, scales = torch.zeros((4, 64), dtype=u8), torch.zeros((4, 2), dtype=u8)
    binding._require(torch.zeros(8, dtype=bf), bf, (8,), cpu, "w")
    binding._require_act8(q.Act8Tensor(codes, scales, (4, 64)), cpu, "x")
    assert binding._rank(torch.zeros((8, 64))) == 8
    refused = [
        lambda: binding._require(None, bf, (8,), cpu, "w"), lambda: binding._require([1.0], bf, (1,), cpu, "w"),
        lambda: binding._require_act8(None, cpu, "x"), lambda: binding._require_act8(codes, cpu, "x"),
        lambda: binding._require_act8(q.Act8Tensor(None, scales, (4, 64)), cpu, "x"),
        lambda: binding._require_act8(q.Act8Tensor(codes, None, (4, 64)), cpu, "x"),
        lambda: binding._require_act8(q.Act8Tensor(codes, scales, (4, 8, 8)), cpu, "x"),
        lambda: binding._require_weight(None, cpu), lambda: binding._require_weight(codes, cpu),
        lambda: binding._require_weight(q.NF4Tensor(None, None, None, None, (64, 64)), cpu),
        lambda: binding._rank(None), lambda: binding._rank(torch.zeros(8)),
        lambda: q.act8_dequant(None), lambda: q.act8_dequant(codes), lambda: q.act8_quantize(None),
        lambda: q.epilogue_bwd(None, None, "silu"), lambda: q.rmsnorm_fwd(None, None),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(q.QNF4Error):
            call()
            pytest.fail(f"call {i} was not refused")
