"""Pins of the block-scaled FP8 oracle: its quantiser against the per-row one
of the W8A8 oracle on rows of one block, its products and norm against
loop-by-loop sums, the SwiGLU against a high-precision evaluation, and the
experts against hand-built weights."""
from fractions import Fraction
import math

import numpy as np
import pytest

from oracle import fp8_block as B
from oracle import formats as F
from oracle import w8a8 as W


def _codes(rng, *shape):
    q = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((q & 0x7F) == 0x7F, 0, q).astype(np.uint8)


def test_quantizer_equals_the_row_quantizer_on_rows_of_one_block():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal((32, 128)) * np.exp2(rng.integers(-20, 20, (32, 1)))).astype(np.float32).astype(np.float64)
    v[3] = 0.0
    q, s = B.quantize(v)
    q2, s2 = W.fp8_quantize(v)
    assert np.array_equal(s[:, 0], s2)
    # the row quantiser rounds v / scale to fp32 first: at most a tie apart
    assert np.mean(q != q2) < 1e-3 and np.all(np.abs(q.astype(int) - q2) <= 1)


def test_partial_last_block_has_its_own_scale():
    v = np.ones((1, 200))
    v[0, 130] = -896.0
    q, s = B.quantize(v)
    assert s.shape == (1, 2) and s[0, 0] == np.float32(1 / 448) and s[0, 1] == 2.0
    assert F.E4M3_TABLE[q[0, 130]] == -448 and F.E4M3_TABLE[q[0, 0]] == 448


def test_linear_equals_exact_sums():
    rng = np.random.default_rng(1)
    xq, wq = _codes(rng, 2, 144), _codes(rng, 130, 144)
    xs, ws = np.exp2(rng.integers(-3, 3, (2, 2))), np.exp2(rng.integers(-3, 3, (2, 2)))
    y, S = B.linear(xq, xs, wq, ws)
    for t, n in ((0, 0), (1, 127), (0, 128), (1, 129)):
        terms = [Fraction(F.E4M3_TABLE[xq[t, k]] * xs[t, k // 128]) * Fraction(F.E4M3_TABLE[wq[n, k]] * ws[n // 128, k // 128])
                 for k in range(144)]
        assert y[t, n] == pytest.approx(float(sum(terms)), rel=1e-12, abs=1e-12 * float(sum(map(abs, terms))))
        assert S[t, n] == pytest.approx(float(sum(map(abs, terms))), rel=1e-12)


def test_norm_and_swiglu_against_math():
    rng = np.random.default_rng(2)
    x, r, gamma = rng.standard_normal((3, 48)), rng.standard_normal((3, 48)), rng.standard_normal(48)
    z, v = B.add_rmsnorm(x, r, gamma, 1e-5)
    for t in range(3):
        m = math.fsum((x[t, i] + r[t, i]) ** 2 for i in range(48)) / 48
        for i in range(48):
            assert v[t, i] == pytest.approx((x[t, i] + r[t, i]) / math.sqrt(m + 1e-5) * gamma[i], rel=1e-13)
    gu = np.array([[-30.0, -1.0, 0.0, 2.0, 1.0, 3.0, 5.0, -4.0]])
    want = [g / (1 + math.exp(-g)) * u for g, u in zip(gu[0, :4], gu[0, 4:])]
    assert np.allclose(B.swiglu(gu)[0], want, rtol=1e-14)


def test_experts_skip_routes_outside_the_rank_and_add_repeated_ones():
    rng = np.random.default_rng(3)
    H, I, E, T = 256, 128, 3, 4
    xq, xs = _codes(rng, T, H), np.full((T, 2), 0.01)
    w13, s13 = _codes(rng, E, 2 * I, H), np.full((E, 2, 2), 1e-3)
    w2, s2 = _codes(rng, E, H, I), np.full((E, 2, 1), 1e-3)
    idx = np.array([[0, 1], [-1, 2], [2, 2], [-1, 7]])
    wts = np.full((T, 2), 0.5)
    out, S, A = B.experts(xq, xs, idx, wts, w13, s13, w2, s2)
    one = lambda t, e: B.mlp(B.rows_value(xq, xs)[t:t + 1], B.weight_value(w13[e], s13[e]), B.weight_value(w2[e], s2[e]))[0][0]
    assert np.allclose(out[0], 0.5 * one(0, 0) + 0.5 * one(0, 1), rtol=1e-12)
    assert np.allclose(out[1], 0.5 * one(1, 2), rtol=1e-12)
    assert np.allclose(out[2], one(2, 2), rtol=1e-12)
    assert np.all(out[3] == 0) and np.all(S[3] == 0) and np.all(A[3] == 0)
    assert np.all(A[:3] >= 0) and np.all(S[:3] > 0)
