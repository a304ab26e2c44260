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
from parity_util import assert_within_tolerance, to_np64

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


# ------------------------------------------------------------------------------- activations
INF = float("inf")


@pytest.mark.parametrize("act", ob.ACTIVATIONS[1:])
def test_epilogue_bwd_at_infinite_pre_activations(act):
    """The slopes' limits, 0 and 1, with a gradient of zero too; a NaN stays one (ReLU's slope at a NaN passes
    the gradient)."""
    z = torch.tensor([-INF, INF, -3.38e38, 3.38e38, -INF, INF, float("nan"), 0.0], dtype=BF).repeat(3, 1)
    dy = torch.tensor([2.0, 2.0, 2.0, 2.0, 0.0, 0.0, 1.0, 0.0], dtype=BF).repeat(3, 1)
    dz, db = q.epilogue_bwd(dy.cuda(), z.cuda(), act, need_dbias=True)
    want = torch.tensor([0.0, 2.0, 0.0, 2.0, 0.0, 0.0, 1.0 if act == "relu" else float("nan"), 0.0]).repeat(3, 1)
    assert _same(dz.float().cpu(), want) and _same(db.float().cpu(), want.sum(dim=0))


@pytest.mark.parametrize("M", [400, 16, 8, 1])
@pytest.mark.parametrize("act", ob.ACTIVATIONS[1:])
def test_activations_over_their_whole_range(act, M):
    """Every pre-activation from -30 to 30 through a layer of one weight, in calls of M tokens, and infinite
    ones through the bias: the formulas' own values, infinite, NaN at -infinity but for ReLU."""
    N, K = 8, 64
    Wm = torch.zeros((N, K), dtype=BF)
    Wm[:, 0] = 1.0
    W = q.nf4_quantize_dq(Wm.cuda())
    assert (q.nf4_dequant(W)[:, 0] == 1).all()
    v = torch.linspace(-30, 30, 400).to(BF)
    x = torch.zeros((400, K), dtype=BF)
    x[:, 0] = v
    x = x.cuda()
    out = torch.cat([q.qlora_linear_epilogue_fwd(x[i:i + M], W, None, None, 1.0, activation=act)[0] for i in range(0, 400, M)])
    zz = np.abs(to_np64(v))[:, None]
    ref = ob.act(to_np64(v)[:, None] * np.ones(N), act)
    # the exponent's argument v = 2 u, rounded, with |v| <= 2 |z| (1 + z^2); below 2^-126 the reciprocal is
    # flushed, so z p is off by |z| 2^-126 at most, and a bf16 result by 2^-134
    bound = (H + (8 + 2 * zz * (1 + zz * zz)) * 2.0 ** -23) * np.abs(ref) + zz * 2.0 ** -126 + 2.0 ** -130
    assert (np.abs(to_np64(out) - ref) <= bound).all()
    ends = torch.tensor([-INF, INF, 0.0, float("nan"), -INF, INF, 1e38, -1e38], dtype=BF)
    y, _, z = q.qlora_linear_epilogue_fwd(torch.zeros((M, K), dtype=BF, device="cuda"), W, None, None, 1.0, bias=ends.cuda(),
                                          activation=act, save=True)
    assert _same(z.cpu(), ends.repeat(M, 1))
    low = 0.0 if act == "relu" else float("nan")
    want = torch.tensor([low, INF, 0.0, float("nan"), low, INF, 1e38, 0.0]).to(BF).repeat(M, 1)
    assert _same(y.cpu(), want)


# ------------------------------------------------------------- rarer routes of a few tokens
def _against_float64(M, N, K, r, act, seed):
    """A call with everything in its epilogue, all outputs against float64 on the dequantized weight (bit-exact
    against the oracle elsewhere); x is scaled so that the products' fp32 sums stay far inside the tolerance's
    floor of 2e-4 (thousands of terms of 2^-4 * 0.02, each addition off by 2^-24 of a sum below 1)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    W = q.nf4_quantize_dq(normal((N, K), 0.02))
    A, B = (normal((r, K), r ** -0.5), normal((N, r), 0.02)) if r else (None, None)
    x, bias, res = normal((M, K), 2.0 ** -4), normal((N,), 0.5), normal((M, N), 2.0)

    def call():
        return q.qlora_linear_epilogue_fwd(x, W, A, B, 0.5, bias=bias, activation=act, residual=res, save=True)

    y, t, z = call()
    again = call()
    torch.cuda.synchronize()
    assert q.check_device_error() == 0 and torch.equal(again[0], y) and torch.equal(again[2], z)
    zr = x.double() @ q.nf4_dequant(W).double().T + bias.double()
    if r:
        tr = 0.5 * (x.double() @ A.double().T)
        zr += tr @ B.double().T
        mag = 0.5 * (x.double().abs() @ A.double().abs().T)
        # a thread's share of K / 256 products in two chains, then 13 additions and the factor
        assert ((t.double() - tr).abs() <= (K / 512 + 20) * U * mag).all()
    zr = zr.cpu().numpy()
    assert_within_tolerance(z, zr, "z")
    assert_within_tolerance(y, ob.act(zr, act) + to_np64(res), "y")


@pytest.mark.parametrize("M,N,K,r", [(1, 5120, 13816, 64), (16, 5120, 13816, 64), (16, 13824, 5112, 8), (9, 13824, 5112, 0),
                                     (8, 5120, 13816, 0)])
def test_ragged_layers_whose_sums_take_several_rounds(M, N, K, r):
    """K % 64 != 0 and more row tiles per SM than the sums of a block have room for: two rounds of tiles (the
    first, third, fourth and last shape), three (the second)."""
    _against_float64(M, N, K, r, "silu", 211)


@pytest.mark.parametrize("M,N,K,r", [(9, 18944, 32008, 16), (16, 18952, 32008, 0), (11, 520, 32008, 16), (5, 136, 64264, 8)])
def test_few_tokens_of_rows_too_long_for_the_few_token_path(M, N, K, r):
    """K % 64 != 0 and rows whose sums do not fit: 16-token tiles, with their epilogue in the tiles where
    N fills the SMs, behind a K split otherwise."""
    _against_float64(M, N, K, r, "gelu", 212)


def test_missing_operands_are_refused():
    x = torch.zeros((8, 64), dtype=BF, device="cuda")
    w, f32 = torch.zeros(64, dtype=BF, device="cuda"), torch.zeros(8, device="cuda")
    W = q.nf4_quantize_dq(_normal((128, 64), 0.02, 1).cuda())
    A, B = torch.zeros((8, 64), dtype=BF, device="cuda"), torch.zeros((128, 8), dtype=BF, device="cuda")
    dY, t, a = torch.zeros((8, 128), dtype=BF, device="cuda"), torch.zeros((8, 8), device="cuda"), q.act8_quantize(x)
    calls = [
        lambda: q.qlora_linear_bwd(dY, a, None, W, A, B, 1.0), lambda: q.qlora_linear_bwd(dY, a, t, W, None, None, 1.0),
        lambda: q.qlora_linear_bwd(dY, a, t, W, A, None, 1.0), lambda: q.qlora_linear_bwd(dY, a, t, None, A, B, 1.0),
        lambda: q.qlora_linear_bwd(dY, a, t, W, A[0], B, 1.0), lambda: q.qlora_linear_bwd(None, a, t, W, A, B, 1.0),
        lambda: q.qlora_linear_epilogue_fwd(x, None, A, B, 1.0), lambda: q.qlora_linear_epilogue_fwd(x, W, A[0], B, 1.0),
        lambda: q.qlora_linear_epilogue_fwd(x, W, 3, B, 1.0), lambda: q.qlora_linear_epilogue_fwd(x, W, A, B, 1.0, bias=0.5),
        lambda: q.rmsnorm_fwd(x, None), lambda: q.rmsnorm_bwd(x, None, f32, w), lambda: q.rmsnorm_bwd(x, x, None, w),
        lambda: q.rmsnorm_bwd(x, x, f32, None), lambda: q.epilogue_bwd(x, 1.0, "silu"),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(q.QNF4Error):
            call()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("M,N,K,r", [(3, 264, 512, 8), (8, 5120, 4096, 16), (9, 264, 512, 0), (16, 1000, 4096, 8), (5, 136, 1000, 8),
                                     (16, 136, 1000, 8), (40, 264, 520, 16), (300, 264, 512, 8)])
def test_tokens_do_not_touch_one_another(M, N, K, r):
    """NaN and infinities in one token's x and residual leave every other token's outputs as they were, bit for
    bit, in a workspace full of NaN as well."""
    inp = synth.linear_inputs(M, N, K, max(r, 8), 221)
    A, B = (inp["A"].cuda(), inp["B"].cuda()) if r else (None, None)
    x, res = inp["x"].cuda(), _normal((M, N), 2.0, 222).cuda()
    W = q.nf4_quantize_dq(_normal((N, K), 0.02, 223).cuda())
    y, _, z = q.qlora_linear_epilogue_fwd(x, W, A, B, 0.5, activation="silu", residual=res, save=True)
    for bad in (0, M // 2, M - 1):
        xb, rb = x.clone(), res.clone()
        xb[bad, ::3], xb[bad, 1::3], rb[bad] = float("nan"), float("inf"), float("-inf")
        ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")
        yb, _, zb = q.qlora_linear_epilogue_fwd(xb, W, A, B, 0.5, activation="silu", residual=rb, save=True, workspace=ws)
        keep = torch.arange(M, device="cuda") != bad
        assert torch.equal(yb[keep], y[keep]) and torch.equal(zb[keep], z[keep])
        assert torch.isnan(yb[bad]).all() and torch.isnan(zb[bad]).all()
    torch.cuda.synchronize()
    assert q.check_device_error() == 0


@pytest.mark.parametrize("M,N,K,r", [(70, 136, 320, 16), (600, 264, 1000, 8), (2100, 128, 256, 64)])
def test_linear_bwd_act8_in_a_workspace_full_of_nan(M, N, K, r):
    """With and without splits of the tokens: nothing is read that the call has not written."""
    inp = synth.linear_inputs(M, N, K, r, 231)
    x, A, B, dY = (inp[k].cuda() for k in ("x", "A", "B", "dY"))
    W = q.nf4_quantize_dq(_normal((N, K), 0.02, 232).cuda())
    _, t = q.qlora_linear_fwd(x, W, A, B, 0.5)
    a = q.act8_quantize(x)
    want = q.qlora_linear_bwd(dY, a, t, W, A, B, 0.5)
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")
    got = q.qlora_linear_bwd(dY, a, t, W, A, B, 0.5, workspace=ws)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
