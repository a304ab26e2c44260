"""Pins of the oracle's operators around the linear: the 8-bit checkpoint format in exact
rationals, the gradients against central differences, the activations' textbook forms."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import block
from oracle.nf4 import bf16_bits_to_f32, e4m3_decode


def _bf16(rng, shape, lo=-130, hi=127):
    """bf16 values whose exponents cover the whole range, as float64."""
    bits = rng.integers(0, 1 << 16, size=shape).astype(np.uint16)
    v = bf16_bits_to_f32(bits).astype(np.float64).reshape(shape)
    return np.where(np.isfinite(v), v, 1.0)


def test_checkpoint_against_exact_rationals():
    rng = np.random.default_rng(1)
    x = _bf16(rng, (24, 72))
    x[3] = 0.0
    x[4, :32] = 448.0 * 2.0 ** -30          # exactly at the boundary, and one bf16 step above it
    x[5, :32] = 452.0 * 2.0 ** -30
    x[6] = rng.standard_normal(72).astype(np.float32).view(np.uint32).__and__(0xFFFF0000).view(np.float32)
    codes, scales = block.act8_quantize(x)
    assert codes.shape == (24, 80) and scales.shape == (24, 3) and not codes[:, 72:].any()
    pos = [Fraction(float(v)) for v in e4m3_decode(np.arange(127, dtype=np.uint8))]
    for i in range(24):
        for g in range(3):
            grp = [Fraction(float(v)) for v in x[i, 32 * g:32 * g + 32]]
            amax = max(abs(v) for v in grp)
            e = -117
            while e < 120 and amax > 448 * Fraction(2) ** e:
                e += 1
            assert int(scales[i, g]) == e + 127
            for j, v in enumerate(grp):
                n = abs(v) / Fraction(2) ** e
                n = min(n, Fraction(240)) if e == 120 else n
                d = [abs(n - q) for q in pos]
                best = min(d)
                ties = [k for k in range(127) if d[k] == best]
                k = ties[0] if len(ties) == 1 else next(k for k in ties if k % 2 == 0)
                assert (int(codes[i, 32 * g + j]) & 0x7F) == k
    back = block.act8_dequant(codes, scales, 72)
    step = np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), 32, axis=1)[:, :72]
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step))


def test_checkpoint_marks_groups_that_are_not_finite():
    x = np.ones((2, 64))
    x[0, 5] = np.inf
    x[1, 40] = np.nan
    codes, scales = block.act8_quantize(x)
    back = block.act8_dequant(codes, scales, 64)
    assert np.isnan(back[0, :32]).all() and (back[0, 32:] == 1).all()
    assert (back[1, :32] == 1).all() and np.isnan(back[1, 32:]).all()


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_gradients_against_differences(with_residual):
    rng = np.random.default_rng(2)
    M, K, eps = 3, 17, 1e-3
    x, w = rng.standard_normal((M, K)), rng.standard_normal(K)
    res = rng.standard_normal((M, K)) if with_residual else None
    dy, dh = rng.standard_normal((M, K)), rng.standard_normal((M, K))

    def loss(x_, w_):
        f = block.rmsnorm_forward(x_, w_, eps, res)
        return (f["y"] * dy).sum() + (f["v"] * dh).sum()

    f = block.rmsnorm_forward(x, w, eps, res)
    b = block.rmsnorm_backward(dy, f["v"], f["rstd"], w, dh)
    t = 1e-6
    for _ in range(20):
        i, k = rng.integers(M), rng.integers(K)
        d = np.zeros((M, K))
        d[i, k] = t
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * t) - b["dx"][i, k]) < 1e-7
        d = np.zeros(K)
        d[k] = t
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * t) - b["dw"][k]) < 1e-7


@pytest.mark.parametrize("name", block.ACTIVATIONS)
def test_slopes_against_differences(name):
    z = np.concatenate([np.linspace(-9, 9, 401) + 0.0123, [-30.0, 30.0]])
    t = 1e-6
    num = (block.act(z + t, name) - block.act(z - t, name)) / (2 * t)
    assert np.all(np.abs(num - block.act_slope(z, name)) < 1e-7)


def test_activations_are_the_textbook_forms():
    z = np.array([-3.0, -0.5, 0.0, 0.7, 2.5])
    assert np.allclose(block.act(z, "silu"), [v / (1 + math.exp(-v)) for v in z], rtol=1e-14)
    assert np.allclose(block.act(z, "gelu"), [0.5 * v * (1 + math.erf(v / math.sqrt(2))) for v in z], rtol=1e-12)
    tanh = [0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))) for v in z]
    assert np.allclose(block.act(z, "gelu_tanh"), tanh, rtol=1e-12)
    assert np.array_equal(block.act(z, "relu"), [0, 0, 0, 0.7, 2.5]) and np.array_equal(block.act(z, "none"), z)
