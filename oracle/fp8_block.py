"""Block-scaled FP8 operators in FP64 (test infrastructure only): E4M3 codes
with one fp32 scale per row and 128 columns, or per 128 x 128 weight block.

    scale = fp32(amax / 448),  code = RNE_E4M3(fp32(v / scale)), saturating;
    a scale that is not positive gives signed zeros.

(The kernels multiply by fp32(1 / scale), which can move a value by a few fp32
units before its rounding: where v / scale lies that near a boundary between two
codes, either is accepted.)

Each function returns the exact result (in float64, from the values the codes
and scales stand for) together with what bounds the error of an fp32
evaluation of it, so that the tests can derive their tolerances.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3_TABLE, e4m3_encode

BLOCK = 128
ACC = 2.0 ** -16     # fp32 accumulation of a dot product, relative to the sum of magnitudes
EPS_H = 2.0 ** -18   # silu(g) * u in fp32 with the hardware exponential, |g| <= 12


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def block_amax(v: np.ndarray) -> np.ndarray:
    """[..., blocks] largest magnitude of each 128-column block of v [..., n]."""
    return np.stack([np.abs(v[..., i:i + BLOCK]).max(-1) for i in range(0, v.shape[-1], BLOCK)], -1)


def spread(s: np.ndarray, n: int) -> np.ndarray:
    """Scales [..., blocks] repeated over the n columns."""
    return np.repeat(np.asarray(s, np.float64), BLOCK, axis=-1)[..., :n]


def quantize(v: np.ndarray):
    """(codes, fp32 scales) of rows v [..., n] by the rule above, in exact arithmetic."""
    s = (block_amax(v) / 448.0).astype(np.float32)
    d = spread(s, v.shape[-1])
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(d > 0, v / d, 0.0 * v)
    return e4m3_encode(t), s


def rows_value(q, s) -> np.ndarray:
    return E4M3_TABLE[np.asarray(q)] * spread(s, np.asarray(q).shape[-1])


def weight_value(q, s) -> np.ndarray:
    """Values of weight codes [..., N, K] with scales [..., N/128, K/128]."""
    q = np.asarray(q)
    N, K = q.shape[-2:]
    return E4M3_TABLE[q] * np.repeat(spread(s, K), BLOCK, axis=-2)[..., :N, :]


def add_rmsnorm(x, residual, gamma, eps):
    """(z, v): the residual stream and its norm times gamma."""
    z = x if residual is None else x + residual
    r = 1.0 / np.sqrt((z * z).sum(-1, keepdims=True) / z.shape[-1] + eps)
    return z, z * r * gamma


def silu(g):
    return g / (1.0 + np.exp(-g))


def swiglu(gu):
    I = gu.shape[-1] // 2
    return silu(gu[..., :I]) * gu[..., I:]


def linear(xq, xs, wq, ws):
    """(y, S): the product and the sum of its terms' magnitudes."""
    x, w = rows_value(xq, xs), weight_value(wq, ws)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def mlp(x, w13, w2):
    """One expert on rows x [n, H] with weight values w13 [2I, H], w2 [H, I]:
    (y, S, A), S the magnitudes of the down product's terms and A how far y may
    move because an fp32 evaluation of h can land on the other side of a
    rounding boundary (or move a scale)."""
    gu, Sgu = x @ w13.T, np.abs(x) @ np.abs(w13).T
    I = w2.shape[1]
    g, u, dg, du = gu[:, :I], gu[:, I:], ACC * Sgu[:, :I], ACC * Sgu[:, I:]
    h = silu(g) * u
    # |silu'| <= 1.1
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + EPS_H * np.abs(h)
    q, s = quantize(h)
    s64 = s.astype(np.float64)
    rel = np.stack([dh[:, i:i + BLOCK].max(-1) for i in range(0, I, BLOCK)], -1) / np.maximum(block_amax(h), 1e-300)
    d, r = spread(s64, I), spread(rel, I) + 2.0 ** -22
    hv = E4M3_TABLE[q] * d
    with np.errstate(divide="ignore", invalid="ignore"):
        lo = E4M3_TABLE[e4m3_encode(np.where(d > 0, (h - dh) / d - np.abs(h / d) * r, 0.0))] * d
        hi = E4M3_TABLE[e4m3_encode(np.where(d > 0, (h + dh) / d + np.abs(h / d) * r, 0.0))] * d
    move = np.maximum(np.abs(hi - hv), np.abs(hv - lo)) + r * np.maximum(np.abs(hi), np.abs(lo))
    return hv @ w2.T, np.abs(hv) @ np.abs(w2).T, move @ np.abs(w2).T


def experts(xq, xs, idx, wts, w13, s13, w2, s2, shared=None):
    """(out, S, A) of the routed experts (indices outside [0, E) skipped) and,
    with shared = (w13, s13, w2, s2), the shared one."""
    T, H = xq.shape
    E = w13.shape[0]
    x = rows_value(xq, xs)
    out, S, A = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))

    def add(t, w, a, b):
        y, s, m = mlp(x[t:t + 1], a, b)
        out[t] += w * y[0]
        S[t] += abs(w) * s[0]
        A[t] += abs(w) * m[0]

    for t in range(T):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if 0 <= e < E:
                add(t, float(wts[t, j]), weight_value(w13[e], s13[e]), weight_value(w2[e], s2[e]))
        if shared is not None:
            add(t, 1.0, weight_value(shared[0], shared[1]), weight_value(shared[2], shared[3]))
    return out, S, A
