"""GPU parity of the operators around the linear (norm, 8-bit checkpoints, epilogue) against the
float64 oracle.

Tolerances.  u = 2^-24 is half an fp32 step, 2^-8 half a bf16 step, both relative.  A sum of n fp32
terms in any order is off by at most n u times the sum of the magnitudes.  The logistic and the
exponential of the activations are within (3 + 1.2 |v|) 2^-23 relative, and their products with the
slope of the argument stay below 2^-17 (|z| u' <= 35 wherever p has not saturated)."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_dq_b200 as q
import synth
from oracle import block as ob
from oracle import linear as olin
from oracle.nf4 import bf16_bits_to_f32
from parity_util import assert_within_tolerance, oracle_weight, to_np64

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def _normal(shape, std, seed):
    return synth.normal_bf16(shape, std, seed)


def _hidden(M, K, seed):
    """Hidden states with a few loud features."""
    v = _normal((M, K), 1.0, seed).float()
    v[:, ::97] *= 20.0
    return v.to(BF)


def _close(got, ref, bound, what):
    g = to_np64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} out of bounds, worst {np.abs(g - ref).max()}"


def _bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


# ------------------------------------------------------------------------ 8-bit checkpoints
SHAPES = [(1, 8), (3, 40), (5, 48), (2, 264), (7, 128), (37, 1000), (2, 13824), (513, 520), (130, 3000)]


def _spread(M, K, seed):
    """bf16 values of every exponent, with rows of zeros, of boundary magnitudes and of subnormals."""
    rng = np.random.default_rng(seed)
    bits = rng.integers(0, 1 << 16, size=(M, K)).astype(np.uint16)
    v = bf16_bits_to_f32(bits).reshape(M, K)
    with np.errstate(invalid="ignore"):
        v = np.where(np.isfinite(v), v, np.float32(1.0))
    x = torch.from_numpy(v.astype(np.float32)).to(BF)
    if M > 2:
        x[0] = 0.0
        x[1, ::3] = 448.0 * 2.0 ** -20
        x[1, 1::3] = 2.0 ** -130
        x[2] = _normal((K,), 1.0, seed + 1)
    return x


@pytest.mark.parametrize("M,K", SHAPES)
def test_act8_is_bit_exact(M, K):
    for x in (_spread(M, K, 3 * M + K), _hidden(M, K, 5)):
        a = q.act8_quantize(x.cuda())
        codes, scales = ob.act8_quantize(to_np64(x))
        assert np.array_equal(a.scales.cpu().numpy(), scales)
        assert np.array_equal(a.codes.cpu().numpy(), codes)
        back = q.act8_dequant(a)
        assert np.array_equal(to_np64(back), ob.act8_dequant(codes, scales, K))
        assert a.nbytes() == codes.size + scales.size


@pytest.mark.parametrize("M,K", [(64, 32), (16, 128), (1, 6144), (4, 13824), (2048, 96), (9480, 2048)])
def test_act8_of_rows_of_whole_groups(M, K):
    """Tensors that make one flat run of rows of 2048 are taken as such; sampled rows of the long one."""
    x = _spread(M, K, M + 7 * K)
    x[M // 2, K - 1] = float("nan")
    a = q.act8_quantize(x.cuda())
    back = q.act8_dequant(a)
    rows = np.arange(M) if M < 4000 else np.r_[0:70, M // 2 - 70:M // 2 + 70, M - 70:M]
    codes, scales = ob.act8_quantize(to_np64(x[rows]))
    group = np.repeat(scales == 255, 32, axis=1)[:, :K]
    assert group.any() and np.array_equal(a.scales.cpu().numpy()[rows], scales)
    assert np.array_equal(a.codes.cpu().numpy()[rows][:, :K][~group], codes[:, :K][~group])
    got = to_np64(back)[rows]
    assert np.isnan(got[group]).all() and np.array_equal(got[~group], ob.act8_dequant(codes, scales, K)[~group])


def test_act8_of_values_that_are_not_finite():
    x = _normal((4, 96), 1.0, 1)
    x[0, 3], x[1, 40], x[2, 95] = float("inf"), float("nan"), float("-inf")
    a = q.act8_quantize(x.cuda())
    _, scales = ob.act8_quantize(to_np64(x))
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    back = to_np64(q.act8_dequant(a))
    group = np.repeat(scales == 255, 32, axis=1)
    assert group.sum() == 96 and np.isnan(back[group]).all() and np.isfinite(back[~group]).all()


def test_act8_offsets_beyond_32_bits():
    M, K = 160001, 13832                       # 2.2e9 values
    x = torch.zeros((M, K), dtype=BF, device="cuda")
    tail = _spread(65, K, 9)
    x[-65:] = tail.cuda()
    a = q.act8_quantize(x)
    codes, scales = ob.act8_quantize(to_np64(tail))
    assert np.array_equal(a.codes[-65:].cpu().numpy(), codes) and np.array_equal(a.scales[-65:].cpu().numpy(), scales)
    del x
    assert np.array_equal(to_np64(q.act8_dequant(a)[-65:]), ob.act8_dequant(codes, scales, K))


# -------------------------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 8), (1, 5120), (3, 40), (7, 264), (37, 1000), (2, 13824), (509, 3000), (130, 4096), (3, 20000),
               (700, 5120)]


def _chain(K):
    """Length of the longest chain of additions in a row sum, generously: one warp, 8 values a step."""
    return 8 * (-(-K // 256)) + 16


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_rmsnorm_fwd(M, K, residual):
    x, w = _hidden(M, K, 11), (1 + 0.1 * _normal((K,), 1.0, 12).float()).to(BF)
    res = _hidden(M, K, 13) if residual else None
    eps = 1e-5
    f = ob.rmsnorm_forward(to_np64(x), to_np64(w), eps, None if res is None else to_np64(res))
    xc, wc, rc = x.cuda(), w.cuda(), None if res is None else res.cuda()
    rel = _chain(K) * U
    for act8 in (False, True):
        y, h, rstd, y8 = q.rmsnorm_fwd(xc, wc, eps=eps, residual=rc, act8=act8)
        _close(rstd, f["rstd"], rel * f["rstd"], "rstd")
        _close(y, f["y"], (H + 2 * rel) * np.abs(f["y"]), "y")
        if residual:
            _close(h, f["v"], (H + U) * np.abs(f["v"]), "h")
        else:
            assert h is xc
        if act8:
            a = q.act8_quantize(y)               # the checkpoint is y's, bit for bit
            assert torch.equal(a.codes, y8.codes) and torch.equal(a.scales, y8.scales) and y8.shape == (M, K)
            assert torch.equal(y, plain[0]) and torch.equal(rstd, plain[1])
        else:
            assert y8 is None
            plain = (y, rstd)


@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_rmsnorm_bwd(M, K, dh):
    h, w = _hidden(M, K, 21), (1 + 0.1 * _normal((K,), 1.0, 22).float()).to(BF)
    dy, e = _normal((M, K), 1.0, 23), _normal((M, K), 1.0, 24) if dh else None
    rstd = torch.rsqrt(h.float().square().mean(dim=1) + 1e-5)
    h64, w64, dy64, r64 = to_np64(h), to_np64(w), to_np64(dy), rstd.numpy().astype(np.float64)
    e64 = None if e is None else to_np64(e)
    b = ob.rmsnorm_backward(dy64, h64, r64, w64, e64)
    n = h64 * r64[:, None]
    g = dy64 * w64
    mag = r64[:, None] * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), axis=1, keepdims=True))
    bound = H * np.abs(b["dx"]) + (_chain(K) + 8) * U * (mag + (0 if e64 is None else np.abs(e64)))
    dwb = H * np.abs(b["dw"]) + (M + 8) * U * np.abs(dy64 * n).sum(axis=0)
    args = (dy.cuda(), h.cuda(), rstd.cuda(), w.cuda())
    ec = None if e is None else e.cuda()
    dx, dw = q.rmsnorm_bwd(*args, dh=ec)
    assert dw is None
    _close(dx, b["dx"], bound, "dx")
    dx, dw = q.rmsnorm_bwd(*args, dh=ec, need_dweight=True)
    _close(dx, b["dx"], bound, "dx with dweight")
    _close(dw, b["dw"], dwb, "dweight")
    again = q.rmsnorm_bwd(*args, dh=ec, need_dweight=True)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)     # no order that changes


def test_rmsnorm_zero_rows_and_large_values():
    x = torch.zeros((3, 64), dtype=BF)
    x[1] = 1e18
    x[2, 0] = 1.0
    w = torch.ones(64, dtype=BF)
    y, h, rstd, y8 = q.rmsnorm_fwd(x.cuda(), w.cuda(), eps=1e-6, act8=True)
    f = ob.rmsnorm_forward(to_np64(x), np.ones(64), 1e-6)
    _close(y, f["y"], (H + 40 * U) * np.abs(f["y"]), "y")
    assert (q.act8_dequant(y8)[0] == 0).all()


def test_rmsnorm_of_rows_whose_squares_overflow():
    """The sum of the squares is fp32: past its range rstd and y are 0, NaN where v is not finite."""
    x = torch.full((2, 64), 1e20, dtype=BF)
    x[1, 5] = float("inf")
    y, _, rstd, _ = q.rmsnorm_fwd(x.cuda(), torch.ones(64, dtype=BF, device="cuda"))
    assert (rstd == 0).all() and (y[0] == 0).all() and torch.isnan(y[1, 5]) and (y[1, 6:] == 0).all()


# --------------------------------------------------------- linear backward from a checkpoint
def _weight(N, K, seed):
    return _normal((N, K), 0.02, seed)


@pytest.mark.parametrize("M,N,K,r", [(1, 128, 64, 8), (65, 256, 512, 16), (130, 520, 1000, 24), (300, 200, 192, 64),
                                     (512, 4096, 4096, 64), (777, 264, 3000, 256), (1030, 1024, 136, 32)])
def test_linear_bwd_act8_equals_the_bf16_pass_on_the_decoded_values(M, N, K, r):
    """Decoding is exact and the products are the same: dA, dB and dX agree bit for bit with the bf16
    pass on the decoded values, and dA with the oracle on them."""
    inp = synth.linear_inputs(M, N, K, r, 31 + M)
    x, A, B, dY = (inp[k].cuda() for k in ("x", "A", "B", "dY"))
    x[0] *= 2.0 ** 40            # scales above 2^7 take the second factor of the decoder
    x[-1] = 0.0
    x[M // 2, ::2] *= 2.0 ** -30
    W = q.nf4_quantize_dq(_weight(N, K, 7).cuda())
    _, t = q.qlora_linear_fwd(x, W, A, B, 0.5)
    a = q.act8_quantize(x)
    xv = q.act8_dequant(a)
    want = q.qlora_linear_bwd(dY, xv, t, W, A, B, 0.5)
    got = q.qlora_linear_bwd(dY, a, t, W, A, B, 0.5)
    torch.cuda.synchronize()
    assert q.check_device_error() == 0
    for g, w_, name in zip(got, want, ("dX", "dA", "dB")):
        assert torch.equal(g, w_), name
    none, dA, dB = q.qlora_linear_bwd(dY, a, t, W, A, B, 0.5, need_dx=False)
    assert none is None and torch.equal(dA, got[1]) and torch.equal(dB, got[2])
    ref = olin.adapter_grads(to_np64(dY), to_np64(xv), to_np64(A), to_np64(B), 0.5)["dA"]
    x64 = np.abs(to_np64(xv))
    u64 = 0.5 * np.abs(to_np64(dY)) @ np.abs(to_np64(B))
    _close(got[1], ref, H * np.abs(ref) + 2.0 ** -14 * (u64.T @ x64), "dA")


def test_linear_bwd_act8_other_formats_and_nan():
    M, N, K, r = 70, 136, 320, 16
    inp = synth.linear_inputs(M, N, K, r, 41)
    x, A, B, dY = (inp[k].cuda() for k in ("x", "A", "B", "dY"))
    for codebook, dq in (("nf4", False), ("fp4_e2m1", True), ("int4", False)):
        W = q.quantize(_weight(N, K, 8).cuda(), codebook, dq)
        _, t = q.qlora_linear_fwd(x, W, A, B, 0.25)
        a = q.act8_quantize(x)
        want = q.qlora_linear_bwd(dY, q.act8_dequant(a), t, W, A, B, 0.25)
        got = q.qlora_linear_bwd(dY, a, t, W, A, B, 0.25)
        assert all(torch.equal(g, w_) for g, w_ in zip(got, want)), codebook
    x[3, 70] = float("nan")
    _, dA, _ = q.qlora_linear_bwd(dY, q.act8_quantize(x), t, W, A, B, 0.25)
    bad = torch.isnan(dA).all(dim=0).cpu()
    assert bad[64:96].all() and not torch.isnan(dA[:, torch.cat((torch.arange(64), torch.arange(96, K))).cuda()]).any()


# ---------------------------------------------------------------------------- linear epilogue
def _epi_ref(x, Wd, A, B, s, bias, act, res):
    z = to_np64(x) @ Wd.T
    t = None
    if A is not None:
        t = s * (to_np64(x) @ to_np64(A).T)
        z = z + t @ to_np64(B).T
    if bias is not None:
        z = z + to_np64(bias)
    y = ob.act(z, act)
    return (y if res is None else y + to_np64(res)), z, t


def _c(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K,r", [(1, 136, 256, 16), (3, 128, 1000, 0), (8, 1024, 512, 8), (9, 264, 520, 16),
                                     (16, 4000, 3000, 8), (17, 256, 192, 64), (48, 520, 1000, 32), (100, 640, 1024, 24),
                                     (300, 200, 192, 64), (600, 1304, 320, 0), (2100, 1152, 256, 8)])
def test_linear_epilogue_fwd(M, N, K, r, act):
    """Token counts of every tile width and of the few-token path, with and without a K split, on
    aligned and K % 64 != 0 weights, with and without adapters."""
    W = _weight(N, K, 51)
    Wd = oracle_weight(W)["w_deq"]
    Wq = q.nf4_quantize_dq(W.cuda())
    inp = synth.linear_inputs(M, N, K, max(r, 8), 52 + M)
    A, B = (inp["A"], inp["B"]) if r else (None, None)
    bias, res = _normal((N,), 0.5, 53), _normal((M, N), 2.0, 54)
    x = inp["x"]
    for use_b, use_r, save in ((True, True, True), (False, False, False), (True, False, False), (False, True, True)):
        b, rs = bias if use_b else None, res if use_r else None
        y, t, z = q.qlora_linear_epilogue_fwd(x.cuda(), Wq, _c(A), _c(B), 0.5, bias=_c(b), activation=act,
                                              residual=_c(rs), save=save)
        torch.cuda.synchronize()
        assert q.check_device_error() == 0
        yr, zr, tr = _epi_ref(x, Wd, A, B, 0.5, b, act, rs)
        assert_within_tolerance(y, yr, f"y {use_b} {use_r}")
        assert (t is not None) == (save and r > 0) and (z is not None) == (save and act != "none")
        if z is not None:
            assert_within_tolerance(z, zr, "z")
        if t is not None:
            mag = 0.5 * (np.abs(to_np64(x)) @ np.abs(to_np64(A)).T)
            _close(t, tr, 128 * 2.0 ** -23 * mag + U * np.abs(tr), "t")


@pytest.mark.parametrize("codebook,dq", [("nf4", False), ("fp4_e2m1", True), ("fp4_e2m1", False), ("int4", True),
                                         ("int4", False)])
def test_linear_epilogue_other_formats(codebook, dq):
    for M, N, K in ((1, 264, 512), (5, 136, 1000), (40, 136, 320), (300, 264, 320)):
        W = q.quantize(_weight(N, K, 61).cuda(), codebook, dq)
        Wd = to_np64(q.nf4_dequant(W))           # bit-exact against the oracle elsewhere
        inp = synth.linear_inputs(M, N, K, 16, 62)
        bias, res = _normal((N,), 0.5, 63), _normal((M, N), 1.0, 64)
        y, _, _ = q.qlora_linear_epilogue_fwd(inp["x"].cuda(), W, inp["A"].cuda(), inp["B"].cuda(), 0.5, bias=bias.cuda(),
                                              activation="silu", residual=res.cuda())
        assert_within_tolerance(y, _epi_ref(inp["x"], Wd, inp["A"], inp["B"], 0.5, bias, "silu", res)[0], f"{M}")


@pytest.mark.parametrize("M,N,K,r", [(1, 5120, 4096, 16), (3, 2376, 3968, 8), (8, 40, 13824, 24), (9, 2376, 3968, 64),
                                     (16, 1000, 20480, 8), (16, 2376, 256, 16), (11, 24, 33024, 0), (2, 1208, 64, 8),
                                     (5, 2376, 2056, 8), (13, 8, 2056, 16)])
def test_few_tokens_joined_in_a_block_and_from_a_flat_list(M, N, K, r):
    """Shapes on both sides of the few-token path's rule: tiles of one block, several rounds of them, a
    flat list whose items cut tiles, a last tile of 8 rows, rows longer than the sums of a block hold,
    rows that are no multiple of 64; sampled outputs against the oracle."""
    W = _weight(N, K, 111)
    Wq = q.nf4_quantize_dq(W.cuda())
    Wd = to_np64(q.nf4_dequant(Wq))              # bit-exact against the oracle elsewhere
    inp = synth.linear_inputs(M, N, K, max(r, 8), 112)
    A, B = (inp["A"], inp["B"]) if r else (None, None)
    x = (inp["x"].float() / 16).to(BF)
    bias, res = _normal((N,), 0.5, 113), _normal((M, N), 2.0, 114)
    y, t, z = q.qlora_linear_epilogue_fwd(x.cuda(), Wq, _c(A), _c(B), 0.5, bias=bias.cuda(), activation="silu",
                                          residual=res.cuda(), save=True)
    again = q.qlora_linear_epilogue_fwd(x.cuda(), Wq, _c(A), _c(B), 0.5, bias=bias.cuda(), activation="silu",
                                        residual=res.cuda())
    torch.cuda.synchronize()
    assert q.check_device_error() == 0 and torch.equal(again[0], y)
    yr, zr, _ = _epi_ref(x, Wd, A, B, 0.5, bias, "silu", res)
    assert_within_tolerance(y, yr, "y")
    assert_within_tolerance(z, zr, "z")


@pytest.mark.parametrize("M,N,K", [(1, 2048, 512), (16, 2376, 3968), (5, 2376, 3968), (9, 2376, 2056)])
def test_few_tokens_on_two_streams_and_in_graphs(M, N, K):
    """Two calls at once, and two captured ones replayed on new tokens: what one call leaves in its
    workspace is never another's."""
    W = q.nf4_quantize_dq(_weight(N, K, 121).cuda())
    inp = synth.linear_inputs(M, N, K, 16, 122)
    A, B, x, res = inp["A"].cuda(), inp["B"].cuda(), inp["x"].cuda(), _normal((M, N), 2.0, 123).cuda()
    other = torch.flip(x, dims=(1,)).contiguous()

    def call(v):
        return q.qlora_linear_epilogue_fwd(v, W, A, B, 0.5, activation="gelu", residual=res)[0]

    want = [call(x).clone(), call(other).clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(call((x, other)[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    held = x.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = call(held)
        graphs.append((g, y))
    held.copy_(other)
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert q.check_device_error() == 0
    assert all(torch.equal(y, want[1]) for _, y in graphs)


def test_linear_epilogue_identity_reproduces_the_weight():
    """x = I without anything behind the product: y = W'^T bit for bit, through the few-token path too."""
    for N, K in ((384, 256), (200, 1000)):
        W = q.nf4_quantize_dq(_weight(N, K, 71).cuda())
        Wd = q.nf4_dequant(W)
        eye = torch.eye(K, dtype=BF, device="cuda")
        y, _, _ = q.qlora_linear_epilogue_fwd(eye, W, None, None, 1.0)
        assert np.array_equal(_bits(y), _bits(Wd.t().contiguous()))
        for m in (1, 2, 7, 8, 16):
            y, _, _ = q.qlora_linear_epilogue_fwd(eye[K - m:].contiguous(), W, None, None, 1.0)
            assert np.array_equal(_bits(y), _bits(Wd.t()[K - m:].contiguous())), m


@pytest.mark.parametrize("M,N,K,r", [(2, 128, 64, 8), (50, 136, 64, 8), (256, 128, 64, 8), (300, 200, 192, 64), (513, 264, 1000, 0), (2100, 1152, 256, 16),
                                     (777, 136, 2048, 32)])
def test_linear_residual_without_an_activation(M, N, K, r):
    """With the product zero (x = 0) y is the residual itself, values that are not finite among it; ragged
    rows and columns, K splits; with a bias too."""
    W = _weight(N, K, 101)
    Wd = oracle_weight(W)["w_deq"]
    Wq = q.nf4_quantize_dq(W.cuda())
    inp = synth.linear_inputs(M, N, K, max(r, 8), 102)
    A, B = (inp["A"].cuda(), inp["B"].cuda()) if r else (None, None)
    x, res, bias = inp["x"], (_normal((M, N), 3.0, 103).float() * 2.0 ** torch.arange(N).remainder(60)).to(BF), _normal((N,), 0.5, 104)
    res[1, 5], res[M - 1, N - 1], res[M // 2, 77] = float("inf"), float("-inf"), float("nan")
    y, _, _ = q.qlora_linear_epilogue_fwd(torch.zeros_like(x).cuda(), Wq, A, B, 0.5, residual=res.cuda())
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=3.0), torch.nan_to_num(res, nan=3.0))
    assert torch.isnan(y).sum() == 1
    for b in (None, bias):
        y, t, _ = q.qlora_linear_epilogue_fwd(x.cuda(), Wq, A, B, 0.5, bias=_c(b), residual=inp["dY"].cuda(), save=True)
        torch.cuda.synchronize()
        assert q.check_device_error() == 0 and (t is not None) == (r > 0)
        A_, B_ = (inp["A"], inp["B"]) if r else (None, None)
        assert_within_tolerance(y, _epi_ref(x, Wd, A_, B_, 0.5, b, "none", inp["dY"])[0], "y")


def test_linear_epilogue_far_tails_of_the_activations():
    """Pre-activations from -30 to 30 and infinite ones, through a one-weight layer."""
    N, K = 8, 64
    Wm = torch.zeros((N, K), dtype=BF)
    Wm[:, 0] = 1.0
    W = q.nf4_quantize_dq(Wm.cuda())
    assert (q.nf4_dequant(W)[:, 0] == 1).all()
    v = torch.linspace(-30, 30, 400).to(BF)
    for M in (400, 1):
        x = torch.zeros((400, K), dtype=BF)
        x[:, 0] = v
        for act in ob.ACTIVATIONS[1:]:
            out = torch.cat([q.qlora_linear_epilogue_fwd(x[i:i + M].cuda(), W, None, None, 1.0, activation=act)[0]
                             for i in range(0, 400 if M > 1 else 8, M)])
            ref = ob.act(to_np64(v)[:len(out), None] * np.ones(N), act)
            zz = np.abs(to_np64(v))[:len(out), None]
            rel = H + (8 + 2 * zz * (1 + zz * zz)) * 2.0 ** -23   # the exponent's argument, rounded, over |v| <= 2 |u|
            # e^-v overflows fp32 above 2^128 and its reciprocal is then 0: z p is off by |z| 2^-128 at most;
            # below that the reciprocal is subnormal, off by 2^-149, and a bf16 result by 2^-134
            _close(out, ref, rel * np.abs(ref) + zz * 2.0 ** -127 + 2.0 ** -130, f"{act} M={M}")


# ---------------------------------------------------------------------- epilogue's gradient
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 264), (33, 256), (130, 1000), (700, 520), (40, 13824)])
def test_epilogue_bwd(M, N, act):
    dy, z = _normal((M, N), 1.0, 81), _normal((M, N), 2.0, 82)
    dy64 = to_np64(dy)
    z8 = q.act8_quantize(z.cuda())
    for zt, zv in ((z.cuda(), z), (z8, q.act8_dequant(z8))):
        slope = ob.act_slope(to_np64(zv), act)
        ref = dy64 * slope
        for need in (False, True):
            dz, db = q.epilogue_bwd(dy.cuda(), zt, act, need_dbias=need)
            _close(dz, ref, H * np.abs(ref) + 2.0 ** -17 * np.abs(dy64), "dz")
            if need:
                bound = (M + 16) * U * np.abs(ref).sum(axis=0) + 2.0 ** -17 * np.abs(dy64).sum(axis=0)
                dbr = ref.sum(axis=0)
                _close(db, dbr, H * np.abs(dbr) + bound, "dbias")
            else:
                assert db is None
    c = q.epilogue_bwd(dy.cuda(), z8, act, need_dbias=True)
    assert torch.equal(c[0], dz) and torch.equal(c[1], db)


def test_epilogue_bwd_extreme_values_stay_finite():
    z = torch.tensor([-3e38, -1e20, -100.0, -0.0, 0.0, 100.0, 1e20, 3e38], dtype=BF).repeat(4, 1)
    dy = torch.ones_like(z)
    want = torch.tensor([0.0, 0, 0, 0.5, 0.5, 1, 1, 1])
    for act in ("silu", "gelu", "gelu_tanh"):
        dz, db = q.epilogue_bwd(dy.cuda(), z.cuda(), act, need_dbias=True)
        assert torch.equal(dz.float().cpu(), want.repeat(4, 1)), act
        assert torch.equal(db.float().cpu(), 4 * want), act
    dz, _ = q.epilogue_bwd(dy.cuda(), z.cuda(), "relu")
    assert torch.equal(dz.float().cpu(), torch.tensor([0.0, 0, 0, 0, 0, 1, 1, 1]).repeat(4, 1))


# ------------------------------------------------------------------------- used together
def _sublayer(x, res, w, W1, A1, B1, b1, W2, A2, B2, dOut, dStream, s):
    """norm -> linear + bias + SiLU -> linear + residual, then all gradients from 8-bit checkpoints."""
    y, h, rstd, y8 = q.rmsnorm_fwd(x, w, residual=res, act8=True)
    g, t1, z1 = q.qlora_linear_epilogue_fwd(y, W1, A1, B1, s, bias=b1, activation="silu", save=True)
    z8, g8 = q.act8_quantize(z1), q.act8_quantize(g)
    out, t2, z2 = q.qlora_linear_epilogue_fwd(g, W2, A2, B2, s, residual=h, save=True)
    assert z2 is None
    dG, dA2, dB2 = q.qlora_linear_bwd(dOut, g8, t2, W2, A2, B2, s)
    dZ, db1 = q.epilogue_bwd(dG, z8, "silu", need_dbias=True)
    dY, dA1, dB1 = q.qlora_linear_bwd(dZ, y8, t1, W1, A1, B1, s)
    dx, dw = q.rmsnorm_bwd(dY, h, rstd, w, dh=dStream, need_dweight=True)
    return {"out": out, "dx": dx, "dw": dw, "db1": db1, "dA1": dA1, "dB1": dB1, "dA2": dA2, "dB2": dB2}


def _sublayer_inputs(M=260, D=512, F=1024, r=16):
    i1, i2 = synth.linear_inputs(M, F, D, r, 91), synth.linear_inputs(M, D, F, r, 92)
    W1, W2 = _weight(F, D, 93), _weight(D, F, 94)
    host = {"x": _normal((M, D), 1.0, 95), "res": _normal((M, D), 1.0, 96),
            "w": (1 + 0.1 * _normal((D,), 1.0, 97).float()).to(BF), "A1": i1["A"], "B1": i1["B"],
            "b1": _normal((F,), 0.3, 98), "A2": i2["A"], "B2": i2["B"], "dOut": i2["dY"],
            "dStream": _normal((M, D), 1.0, 99)}
    dev = {k: v.cuda() for k, v in host.items()}
    dev["W1"], dev["W2"], dev["s"] = q.nf4_quantize_dq(W1.cuda()), q.nf4_quantize_dq(W2.cuda()), 0.5
    return host, dev, oracle_weight(W1)["w_deq"], oracle_weight(W2)["w_deq"]


def test_a_sublayer_forward_and_backward():
    """The whole chain against float64.  The checkpoints hold 4 significant bits: an element of them is
    off by up to 2^-4 of itself, independently from element to element, which over sums of many
    leaves a few per cent (3 sigma of 2^-4 / sqrt(3) / sqrt(n) plus the slope's own change through z);
    the gradients' norms are held to 2^-4."""
    host, dev, Wd1, Wd2 = _sublayer_inputs()
    got = _sublayer(**dev)
    torch.cuda.synchronize()
    assert q.check_device_error() == 0
    h = {k: to_np64(v) for k, v in host.items()}
    s = 0.5
    f = ob.rmsnorm_forward(h["x"], h["w"], 1e-5, h["res"])
    t1 = s * f["y"] @ h["A1"].T
    z = f["y"] @ Wd1.T + t1 @ h["B1"].T + h["b1"]
    g = ob.act(z, "silu")
    t2 = s * g @ h["A2"].T
    out = g @ Wd2.T + t2 @ h["B2"].T + f["v"]
    dO = h["dOut"]
    b2 = olin.qlora_backward(dO, g, Wd2, h["A2"], h["B2"], s)
    dz = b2["dX"] * ob.act_slope(z, "silu")
    b1 = olin.qlora_backward(dz, f["y"], Wd1, h["A1"], h["B1"], s)
    n = ob.rmsnorm_backward(b1["dX"], f["v"], f["rstd"], h["w"], h["dStream"])
    ref = {"out": out, "dx": n["dx"], "dw": n["dw"], "db1": dz.sum(axis=0), "dA1": b1["dA"], "dB1": b1["dB"],
           "dA2": b2["dA"], "dB2": b2["dB"]}
    for k, v in ref.items():
        off = np.linalg.norm(to_np64(got[k]) - v) / np.linalg.norm(v)
        assert off <= (2.0 ** -6 if k == "out" else 2.0 ** -4), (k, off)


def test_a_sublayer_on_another_stream_and_in_a_graph():
    _, dev, _, _ = _sublayer_inputs(M=70)
    want = {k: v.clone() for k, v in _sublayer(**dev).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _sublayer(**dev)
    side.synchronize()
    assert all(torch.equal(other[k], want[k]) for k in want)
    # two graphs whose workspaces the allocator may share, replayed in turn on new inputs
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_sublayer(**dev))
        graphs.append(g)
    dev["x"].copy_(torch.flip(dev["x"], dims=(0,)))
    new = {k: v.clone() for k, v in _sublayer(**dev).items()}
    assert not torch.equal(new["out"], want["out"])
    for _ in range(3):
        for g, o in zip(graphs, outs):
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[k], new[k]) for k in new)


def test_refusals_with_gpu_operands():
    x = torch.zeros((8, 64), dtype=BF, device="cuda")
    w = torch.zeros(64, dtype=BF, device="cuda")
    W = q.nf4_quantize_dq(_weight(128, 64, 1).cuda())
    A, B = torch.zeros((8, 64), dtype=BF, device="cuda"), torch.zeros((128, 8), dtype=BF, device="cuda")
    f32 = torch.zeros(8, device="cuda")
    calls = [
        lambda: q.act8_quantize(x.float()), lambda: q.act8_quantize(x.t()), lambda: q.act8_quantize(x[:, :60]),
        lambda: q.act8_quantize(x[:, :60].contiguous()), lambda: q.act8_quantize(x[:0]),
        lambda: q.act8_quantize(x.view(-1)[1:505].view(8, 63)),
        lambda: q.act8_quantize(x.view(-1)[1:505 - 56].view(7, 64)),           # a base that is not 16-byte aligned
        lambda: q.act8_dequant(q.Act8Tensor(x.view(torch.uint8), x.view(torch.uint8), (8, 64))),
        lambda: q.rmsnorm_fwd(x, w[:56]), lambda: q.rmsnorm_fwd(x, w, eps=-1.0),
        lambda: q.rmsnorm_fwd(x, w, residual=x[:4]), lambda: q.rmsnorm_fwd(x, w.cpu()),
        lambda: q.rmsnorm_bwd(x, x, f32[:4], w), lambda: q.rmsnorm_bwd(x, x, f32.double(), w),
        lambda: q.rmsnorm_bwd(x, x, f32, w, dh=x[:1]),
        lambda: q.qlora_linear_epilogue_fwd(x, W, A, None, 1.0), lambda: q.qlora_linear_epilogue_fwd(x, W, A, A, 1.0),
        lambda: q.qlora_linear_epilogue_fwd(x[:, :56].contiguous(), W, A, B, 1.0),
        lambda: q.qlora_linear_epilogue_fwd(x, W, A, B, 1.0, bias=w),
        lambda: q.qlora_linear_epilogue_fwd(x, W, A, B, 1.0, residual=x),
        lambda: q.qlora_linear_epilogue_fwd(x, W, A, B, 1.0, activation="swish"),
        lambda: q.qlora_linear_epilogue_fwd(x, q.NF4Tensor(W.codes[:100], W.scale_codes, W.c2, W.mean, (128, 64)), A, B, 1.0),
        lambda: q.epilogue_bwd(x, None, "silu"), lambda: q.epilogue_bwd(x, x[:4], "silu"),
        lambda: q.epilogue_bwd(x, q.act8_quantize(x[:4].contiguous()), "silu"),
        lambda: q.qlora_linear_bwd(torch.zeros((8, 128), dtype=BF, device="cuda"), q.act8_quantize(x[:4].contiguous()),
                                   torch.zeros((8, 8), device="cuda"), W, A, B, 1.0),
        lambda: q.qlora_linear_bwd(torch.zeros((8, 128), device="cuda"), q.act8_quantize(x),
                                   torch.zeros((8, 8), device="cuda"), W, A, B, 1.0),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(q.QNF4Error):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
