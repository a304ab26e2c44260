"""Calls of the operators around the linear that lie beside the ordinary ones: checkpoints whose codes
come from elsewhere, infinite pre-activations, shapes that take the rarer routes of the few-token
path, operands that are missing.

Tolerances as in test_gpu_block.py: u = 2^-24 is half an fp32 step, 2^-8 half a bf16 step."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_dq_b200 as q
import synth
from oracle import block as ob
from parity_util import to_np64

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def _same(a, b):
    """Equal values, NaN where the other has NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def _normal(shape, std, seed):
    return synth.normal_bf16(shape, std, seed)


# ------------------------------------------------------------------------ 8-bit checkpoints
@pytest.mark.parametrize("first", range(0, 256, 8))
def test_act8_decoders_agree_on_every_code_and_scale_byte(first):
    """Eight rows of all 256 codes, one scale byte each: the values are those of the format, rounded to
    bf16, and the backward passes that decode on chip take the same values."""
    M, K, N, r = 8, 256, 128, 8
    codes = torch.arange(256, dtype=torch.uint8).repeat(M, 1)
    scales = torch.arange(first, first + 8, dtype=torch.uint8)[:, None].repeat(1, K // 32)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(ob.act8_dequant(codes.numpy(), scales.numpy(), K).astype(np.float32)).to(BF)
    a = q.Act8Tensor(codes.cuda(), scales.cuda(), (M, K))
    d = q.act8_dequant(a)
    assert _same(d.cpu(), want)
    ones = torch.ones((M, K), dtype=BF, device="cuda")
    assert _same(q.epilogue_bwd(ones, a, "silu")[0], q.epilogue_bwd(ones, d, "silu")[0])
    inp = synth.linear_inputs(M, N, K, r, 201)
    A, B, dY = (inp[k].cuda() for k in ("A", "B", "dY"))
    W = q.nf4_quantize_dq(_normal((N, K), 0.02, 202).cuda())
    t = torch.ones((M, r), device="cuda")
    dX, dA, dB = q.qlora_linear_bwd(dY, a, t, W, A, B, 0.5)
    want = q.qlora_linear_bwd(dY, d, t, W, A, B, 0.5)
    assert torch.equal(dX, want[0]) and _same(dA, want[1]) and torch.equal(dB, want[2])
    assert torch.isnan(dA[:, 127]).all() and torch.isnan(dA[:, 255]).all()
