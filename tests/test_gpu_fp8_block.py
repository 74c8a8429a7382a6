"""GPU parity of the block-scaled FP8 operators against the FP64 oracle.

Tolerances, fixed before the first run:
  * norm: v within 2^-16 |v| in fp32 (a sum of squares of at most a hundred
    fp32 additions in depth, a reciprocal square root, three products), then
    one bf16 rounding (2^-9); codes: one of those the quantiser gives for
    t (1 +- 2^-15), t the exact v / scale; scales within 2^-15;
  * SwiGLU: 2^-18 |h| (the hardware exponential's 2 + 1.2 |g| units in the
    last place, |g| <= 12), codes and scales as above;
  * products: 2^-16 of the sum of the terms' magnitudes (fp32 accumulation),
    then one rounding to the output type;
  * experts: as products, plus how far the output moves where the fp32 h can
    land on the other side of a rounding boundary.
"""
import numpy as np
import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
from oracle import formats as F
from oracle import fp8_block as B

from gpu_util import ensure_built, to_np, torch_cuda

pytestmark = pytest.mark.gpu

U_BF16, U_F32 = 2.0 ** -8 * (1 + 2.0 ** -8), 2.0 ** -24  # half a unit in the last of 8 and 24 bits


@pytest.fixture(scope="module")
def ops():
    torch_cuda()
    ensure_built()
    from block_scaled_fp4_sigmoid_gb300 import fp8_block
    return fp8_block


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(a):
    """(tensor, float64 values) of a rounded to bf16."""
    import torch
    t = torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def f64(t):
    return to_np(t.double())


def check_codes(q, s, v, delta=2.0 ** -15):
    """Codes q and scales s of exact values v."""
    want = B.block_amax(v) / 448.0
    assert np.all(np.abs(s - want) <= delta * want + 2.0 ** -149)
    d = B.spread(want, v.shape[-1])
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(d > 2.0 ** -126, v / d, 0.0 * v)
    a = F.E4M3_TABLE[F.e4m3_encode(t * (1 - delta))]
    b = F.E4M3_TABLE[F.e4m3_encode(t * (1 + delta))]
    g = F.E4M3_TABLE[q]
    bad = ~((np.minimum(a, b) <= g) & (g <= np.maximum(a, b))) & (d > 2.0 ** -126)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    assert np.array_equal(np.signbit(g)[t != 0], np.signbit(t)[t != 0])


# ------------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,H", [(1, 16), (1, 7168), (3, 144), (37, 2000), (130, 1024), (5, 16400), (2, 40000),
                                 (1, 65536)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(ops, T, H, residual):
    rng = np.random.default_rng(T + H)
    x, xv = bf16(rng.standard_normal((T, H)) * np.exp2(rng.integers(-8, 8, (T, 1))))
    r, rv = bf16(rng.standard_normal((T, H))) if residual else (None, None)
    gamma, gv = bf16(1 + 0.2 * rng.standard_normal(H))
    res, y, q, s = ops.add_rmsnorm_fp8(x, r, gamma, 1e-6, want_y=True)
    z, v = B.add_rmsnorm(xv, rv, gv, 1e-6)
    assert np.all(np.abs(f64(res) - z) <= U_BF16 * np.abs(z) + 2.0 ** -133)
    assert (res is x) == (not residual)
    assert np.all(np.abs(f64(y) - v) <= (U_BF16 + 2.0 ** -16) * np.abs(v) + 2.0 ** -133)
    check_codes(to_np(q), f64(s), v)


def test_norm_strided_rows_in_place_and_without_codes(ops):
    import torch
    rng = np.random.default_rng(1)
    T, H = 9, 528
    wide, wv = bf16(rng.standard_normal((T, H + 24)))
    x, xv = wide[:, 8:8 + H], wv[:, 8:8 + H]
    r, rv = bf16(rng.standard_normal((T, H)))
    gamma, gv = bf16(np.ones(H))
    z, v = B.add_rmsnorm(xv, rv, gv, 1e-5)
    want = ops.add_rmsnorm_fp8(x.contiguous(), r, gamma, 1e-5, want_y=True)
    res, y, q, s = ops.add_rmsnorm_fp8(x, r, gamma, 1e-5, residual_out=r, want_y=True)  # r updated in place
    assert res is r
    for a, b in zip((res, y, q, s), want):
        assert torch.equal(a, b)
    assert np.all(np.abs(f64(res) - z) <= U_BF16 * np.abs(z) + 2.0 ** -133)
    y2 = torch.empty_like(y)
    fm.add_rmsnorm_fp8(want[0].data_ptr(), H, None, gamma.data_ptr(), T, H, 1e-5, None, y2.data_ptr(), None, None)
    torch.cuda.synchronize()
    zb = f64(want[0])
    v2 = B.add_rmsnorm(zb, None, gv, 1e-5)[1]
    assert np.all(np.abs(f64(y2) - v2) <= (U_BF16 + 2.0 ** -16) * np.abs(v2) + 2.0 ** -133)


def test_norm_zero_rows_and_values_that_are_not_finite(ops):
    rng = np.random.default_rng(2)
    T, H = 6, 272
    a = rng.standard_normal((T, H))
    a[1] = 0.0
    a[2, 5] = np.nan
    a[3, 200] = np.inf
    x, xv = bf16(a)
    gamma, gv = bf16(np.ones(H))
    _, y, q, s = ops.add_rmsnorm_fp8(x, None, gamma, 0.0, want_y=True)
    y, q, s = f64(y), F.E4M3_TABLE[to_np(q)], f64(s)
    # the zero row: 0 * rsqrt(0) is NaN by the formula with eps = 0
    assert np.all(np.isnan(y[1])) and np.all(np.isnan(s[1]))
    assert np.all(np.isnan(y[2])) and np.all(np.isnan(q[2])) and np.all(np.isnan(s[2]))
    # an infinity: rsqrt(inf) = 0, so its own column is NaN, the others 0
    assert np.isnan(y[3, 200]) and np.all(np.delete(y[3], 200) == 0)
    assert np.isnan(s[3, 1]) and s[3, 0] == 0 and np.all(q[3, :128] == 0) and np.isnan(q[3, 200])
    rest = [0, 4, 5]
    check_codes(to_np(ops.add_rmsnorm_fp8(x, None, gamma, 0.0)[2])[rest], s[rest], B.add_rmsnorm(xv[rest], None, gv, 0.0)[1])
    _, y, q, s = ops.add_rmsnorm_fp8(x, None, gamma, 1e-6, want_y=True)
    assert np.all(f64(y)[1] == 0) and np.all(f64(s)[1] == 0) and np.all((to_np(q)[1] & 0x7F) == 0)


# ---------------------------------------------------------------------- SwiGLU
@pytest.mark.parametrize("T,I,pad", [(1, 16, 0), (8, 2048, 0), (3, 1552, 32), (131, 144, 8), (2, 65536, 0)])
def test_swiglu(ops, T, I, pad):
    rng = np.random.default_rng(T + I)
    gu, v = bf16(np.clip(rng.standard_normal((T, 2 * I + pad)) * 3, -12, 12))
    q, s = ops.swiglu_fp8(gu[:, :2 * I])
    check_codes(to_np(q), f64(s), B.swiglu(v[:, :2 * I]))


def test_swiglu_extremes(ops):
    import torch
    I = 256
    g = np.zeros((4, 2 * I))
    g[0, :I], g[0, I:] = -200.0, 3.0       # e^200 overflows: h = -0
    g[1, :I], g[1, I:] = 200.0, 3.0        # silu(g) = g
    g[2, 7] = np.nan
    g[2, I:] = 1.0
    g[3, :I], g[3, I:] = np.inf, 1.0
    gu, _ = bf16(g)
    q, s = ops.swiglu_fp8(gu)
    q, s = F.E4M3_TABLE[to_np(q)], f64(s)
    assert np.all(q[0] == 0) and np.all(s[0] == 0)
    assert np.all(q[1] == 448) and np.allclose(s[1], 600 / 448, rtol=2.0 ** -20)
    assert np.isnan(s[2, 0]) and s[2, 1] == 0 and np.isnan(q[2, 7]) and np.all(np.delete(q[2], 7) == 0)
    assert np.all(np.isinf(s[3])) and np.all(np.isnan(q[3]))
    assert torch.isfinite(gu[1]).all()


# ---------------------------------------------------------------------- linear
def codes(rng, *shape):
    q = F.e4m3_encode(np.clip(rng.standard_normal(shape) * 110, -448, 448))
    return q


def linear_inputs(T, K, N, seed):
    rng = np.random.default_rng(seed)
    kb = B.blocks(K)
    return (codes(rng, T, K), (0.01 * (0.5 + rng.random((T, kb)))).astype(np.float32), codes(rng, N, K),
            (2e-4 * (0.5 + rng.random((B.blocks(N), kb)))).astype(np.float32))


SHAPES = [(1, 16, 1), (1, 7168, 576), (7, 256, 65), (8, 144, 128), (9, 1040, 130), (16, 2048, 272), (17, 512, 257),
          (31, 400, 100), (33, 1024, 513), (64, 2064, 64), (65, 128, 384), (128, 640, 256), (129, 1536, 1000),
          (200, 272, 31), (300, 512, 768), (513, 896, 515), (1025, 384, 640), (40, 48, 130), (150, 48, 130),
          (140, 2704, 300), (257, 2704, 1100), (513, 2704, 1200), (1024, 1024, 7168), (1030, 1040, 7101)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear(ops, T, K, N, fp32):
    import torch
    xq, xs, wq, ws = linear_inputs(T, K, N, T + K + N)
    y, S = B.linear(xq, xs, wq, ws)
    a = [dev(v) for v in (xq, xs, wq, ws)]
    sc = torch.full((fm.linear_fp8_block_workspace_size(T, K, N),), 0xA5, dtype=torch.uint8, device="cuda")
    got = ops.linear_fp8_block(*a, out_dtype=torch.float32 if fp32 else torch.bfloat16, ws=sc)
    assert fm.get_status(sc.data_ptr()) == (0, 0)
    bad = np.abs(f64(got) - y) > (U_F32 if fp32 else U_BF16) * np.abs(y) + B.ACC * S
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    again = ops.linear_fp8_block(*a, out_dtype=got.dtype)
    assert torch.equal(got, again)


@pytest.mark.parametrize("T,K,N", [(3, 256, 48), (40, 512, 200), (300, 384, 520)])
def test_linear_writes_its_columns_of_a_wider_output_only(ops, T, K, N):
    import torch
    a = [dev(v) for v in linear_inputs(T, K, N, 5)]
    want = ops.linear_fp8_block(*a)
    wide = torch.full((T + 1, N + 37), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.linear_fp8_block(*a, out=wide[:T, 3:3 + N])
    assert torch.equal(wide[:T, 3:3 + N], want)
    wide[:T, 3:3 + N] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,K,N", [(20, 256, 100), (300, 384, 523), (1030, 1040, 7100), (1024, 1024, 7168), (140, 2704, 300)])
def test_linear_into_aligned_columns_of_a_wider_output(ops, T, K, N, fp32):
    """As above with rows and first column on 16 bytes, where whole boxes are stored: their
    parts outside [T, N] stay as they were."""
    import torch
    dtype = torch.float32 if fp32 else torch.bfloat16
    a = [dev(v) for v in linear_inputs(T, K, N, 5)]
    want = ops.linear_fp8_block(*a, out_dtype=dtype)
    wide = torch.full((T + 33, (N + 90) // 8 * 8), 7.0, dtype=dtype, device="cuda")
    ops.linear_fp8_block(*a, out=wide[:T, 8:8 + N])
    assert torch.equal(wide[:T, 8:8 + N], want)
    wide[:T, 8:8 + N] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("at", [0, 1, 6])
@pytest.mark.parametrize("T,K,N", [(40, 14336, 291), (130, 2048, 811), (257, 4096, 1501), (200, 4096, 4099), (163, 576, 2925),
                                   (9, 1024, 8191), (600, 512, 5001), (70, 2048, 1029),
                                   (5, 512, 24571)])
def test_linear_rows_that_start_anywhere(ops, T, K, N, at, fp32):
    """Odd widths, first columns off 16 bytes, few rows in the last tile: tiles of one CTA and of
    clusters of two, four and eight, against 64 bits; nothing else is written."""
    import torch
    xq, xs, wq, ws = linear_inputs(T, K, N, T + N)
    y, S = B.linear(xq, xs, wq, ws)
    wide = torch.full((T + 2, N + at + 5), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    ops.linear_fp8_block(*[dev(v) for v in (xq, xs, wq, ws)], out=wide[1:T + 1, at:at + N])
    bad = np.abs(f64(wide[1:T + 1, at:at + N]) - y) > (U_F32 if fp32 else U_BF16) * np.abs(y) + B.ACC * S
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    wide[1:T + 1, at:at + N] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("T,K,N", [(2, 256, 40), (40, 384, 300), (260, 512, 300)])
def test_linear_nan_stays_in_its_row_and_column(ops, T, K, N):
    xq, xs, wq, ws = linear_inputs(T, K, N, 6)
    xq[1, 130] = 0x7F
    wq[17, 255] = 0xFF
    xs[0, 1] = np.inf
    got = f64(ops.linear_fp8_block(*[dev(v) for v in (xq, xs, wq, ws)]))
    assert np.all(np.isnan(got[1])) and np.all(np.isnan(got[:, 17]))
    assert not np.isfinite(np.delete(got[0], 17)).any()
    rest = np.delete(np.delete(got, [0, 1], 0), 17, 1)
    assert np.isfinite(rest).all()


def test_linear_rows_do_not_depend_on_the_batch_around_them(ops):
    """A token's result at the sizes where the kernel is chosen by T stays within the bound of
    every other batch's, and zero scales give exact zeros."""
    xq, xs, wq, ws = linear_inputs(300, 640, 384, 8)
    xs[4] = 0.0
    y, S = B.linear(xq[:1], xs[:1], wq, ws)
    for T in (5, 16, 32, 33, 64, 128, 300):
        got = f64(ops.linear_fp8_block(*[dev(v) for v in (xq[:T], xs[:T], wq, ws)]))
        assert np.all(np.abs(got[:1] - y) <= U_BF16 * np.abs(y) + B.ACC * S), T
        assert np.all(got[4] == 0), T


def test_linear_on_another_stream_and_in_a_graph(ops):
    import torch
    T, K, N = 150, 512, 640
    a = [dev(v) for v in linear_inputs(T, K, N, 9)]
    want = ops.linear_fp8_block(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ops.linear_fp8_block(*a)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    ws = torch.empty(fm.linear_fp8_block_workspace_size(T, K, N), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.linear_fp8_block(*a, out=out, ws=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("T,K,N", [(4096, 7168, 2112), (1000, 18432, 1024)])
def test_linear_full_size_on_sampled_rows(ops, T, K, N):
    import torch
    rng = np.random.default_rng(3)
    xq, xs, wq, ws = linear_inputs(T, K, N, 10)
    got = f64(ops.linear_fp8_block(*[dev(v) for v in (xq, xs, wq, ws)], out_dtype=torch.float32))
    rows = np.unique(np.r_[0, T - 1, rng.integers(0, T, 24)])
    y, S = B.linear(xq[rows], xs[rows], wq, ws)
    assert np.all(np.abs(got[rows] - y) <= U_F32 * np.abs(y) + B.ACC * S)


# --------------------------------------------------------------------- experts
def expert_inputs(T, H, I, E, k, seed, shared=False, outside=0.0, repeat=False):
    rng = np.random.default_rng(seed)
    hb, ib = H // 128, I // 128
    sc = lambda *s: (2e-4 * (0.5 + rng.random(s))).astype(np.float32)  # noqa: E731
    xq, xs = codes(rng, T, H), (0.01 * (0.5 + rng.random((T, hb)))).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < outside] = -1
    if repeat and k > 1:
        idx[:, 1] = idx[:, 0]
    wts = (0.1 + rng.random((T, k))).astype(np.float32)
    w = [codes(rng, E, 2 * I, H), sc(E, 2 * ib, hb), codes(rng, E, H, I), sc(E, hb, ib)]
    sh = [codes(rng, 2 * I, H), sc(2 * ib, hb), codes(rng, H, I), sc(hb, ib)] if shared else []
    return xq, xs, idx, wts, w, sh


EXPERTS = [dict(T=1, H=256, I=128, E=4, k=1), dict(T=1, H=1024, I=384, E=16, k=8, shared=True),
           dict(T=8, H=512, I=256, E=32, k=4), dict(T=9, H=768, I=128, E=6, k=6, shared=True),
           dict(T=16, H=512, I=256, E=48, k=8, outside=0.7), dict(T=5, H=256, I=256, E=9, k=3, repeat=True),
           dict(T=16, H=256, I=128, E=512, k=16, shared=True), dict(T=3, H=256, I=128, E=1, k=1),
           dict(T=3, H=5120, I=128, E=4, k=2), dict(T=12, H=5120, I=384, E=5, k=3, shared=True),
           # gate/up units shared by eight, four and two CTAs, and by two in several rounds
           dict(T=1, H=4096, I=128, E=4, k=1), dict(T=3, H=2048, I=384, E=6, k=2), dict(T=4, H=4096, I=512, E=16, k=4),
           dict(T=2, H=2304, I=256, E=3, k=2, shared=True), dict(T=16, H=5120, I=640, E=12, k=12),
           # output columns shared by four and two CTAs
           dict(T=7, H=512, I=1024, E=24, k=6, shared=True), dict(T=16, H=1024, I=768, E=24, k=6, outside=0.3)]


@pytest.mark.parametrize("c", EXPERTS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_experts(ops, c):
    import torch
    xq, xs, idx, wts, w, sh = expert_inputs(seed=11, **c)
    ref, S, A = B.experts(xq, xs, idx, wts, *w, shared=sh or None)
    a = [dev(v) for v in (xq, xs, idx, wts, *w, *sh)]
    got = ops.experts_fp8_block(*a)
    bad = np.abs(f64(got) - ref) > U_BF16 * (np.abs(ref) + A) + B.ACC * S + A
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    assert torch.equal(got, ops.experts_fp8_block(*a))


def test_experts_of_masked_tokens_and_nan_weights(ops):
    """A token without routes gives zeros whatever the buffers hold, and an expert of NaN
    weights reaches its own tokens only."""
    import torch
    T, H, I, E, k = 12, 256, 128, 8, 2
    xq, xs, idx, wts, w, _ = expert_inputs(T, H, I, E, k, 12)
    idx[:] = np.arange(T)[:, None] % 4 + np.array([0, 1])
    idx[3] = -1
    idx[7] = [E, 600]
    idx[5] = [7, 6]
    w[0][7] = 0x7F  # expert 7: only token 5
    w[2][7] = 0xFF
    a = [dev(v) for v in (xq, xs, idx, wts, *w)]
    dims = fm.make_dims(T, H, I, E, k, fmt=fm.FP8)
    ws = torch.full((fm.experts_fp8_block_workspace_size(dims),), 0xFF, dtype=torch.uint8, device="cuda")
    got = f64(ops.experts_fp8_block(*a, ws=ws))
    assert np.all(got[[3, 7]] == 0) and np.all(np.isnan(got[5]))
    assert np.isfinite(np.delete(got, 5, 0)).all()
    idx[:] = -1
    assert np.all(f64(ops.experts_fp8_block(*[dev(v) for v in (xq, xs, idx, wts, *w)], ws=ws)) == 0)


def test_experts_on_another_stream_after_the_router(ops):
    """The sublayers run the operators in order on the current stream: equal to the single calls."""
    import torch
    T, H, I, E, k = 6, 512, 256, 16, 4
    _, _, _, _, w, sh = expert_inputs(T, H, I, E, k, 13, shared=True)
    rng = np.random.default_rng(14)
    x, r = bf16(rng.standard_normal((T, H)))[0], bf16(rng.standard_normal((T, H)))[0]
    gamma, wr = bf16(np.ones(H))[0], bf16(rng.standard_normal((E, H)) * 0.05)[0]
    bias = dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    dims = fm.make_dims(T, H, I, E, k, n_shared=1, routed_scaling=2.5, fmt=fm.FP8)
    wd, sd = [dev(v) for v in w], [dev(v) for v in sh]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        moe = ops.Fp8BlockMoE(dims, gamma, wr, bias, *wd, *sd)
        out, res = moe.forward(x, r)
        mlp_out, mlp_res = ops.Fp8BlockMlp(gamma, *sd).forward(out, res)
    s.synchronize()
    res2, y, q, sc = ops.add_rmsnorm_fp8(x, r, gamma, 1e-6, want_y=True)
    idx, tw = moe.route(y)
    want = ops.experts_fp8_block(q, sc, idx, tw, *wd, *sd)
    assert torch.equal(out, want) and torch.equal(res, res2)
    assert bool((idx >= 0).all()) and np.allclose(f64(tw).sum(1), 2.5, rtol=1e-5)
    # the MLP of the shared expert's weights: the same as a layer of it alone
    mr, _, mq, ms = ops.add_rmsnorm_fp8(want, res2, gamma, 1e-6)
    hq, hs = ops.swiglu_fp8(ops.linear_fp8_block(mq, ms, sd[0], sd[1]))
    assert torch.equal(mlp_out, ops.linear_fp8_block(hq, hs, sd[2], sd[3])) and torch.equal(mlp_res, mr)


@pytest.mark.parametrize("T,H,I", [(6, 1024, 640), (130, 1024, 3584), (1024, 1024, 3584), (700, 2816, 256)])
def test_calls_in_a_row_equal_calls_that_wait(ops, T, H, I):
    """Each kernel starts while the one before it ends: a chain of calls that nothing waits
    between, on rotating buffers, gives what the same calls give one by one (streamed, tiled,
    split over clusters, and two launches a product)."""
    import torch
    rng = np.random.default_rng(T)
    w13, s13 = dev(codes(rng, 2 * I, H)), dev((2e-4 * (0.5 + rng.random((2 * I // 128, B.blocks(H))))).astype(np.float32))
    w2, s2 = dev(codes(rng, H, I)), dev((2e-4 * (0.5 + rng.random((B.blocks(H), B.blocks(I))))).astype(np.float32))
    gamma = bf16(np.ones(H))[0]
    xs = [bf16(rng.standard_normal((T, H)))[0] for _ in range(3)]

    def step(x, res, sync):
        out = []
        res, _, q, s = ops.add_rmsnorm_fp8(x, res, gamma, 1e-6)
        for f in (lambda: ops.linear_fp8_block(q, s, w13, s13), lambda: ops.swiglu_fp8(out[0]),
                  lambda: ops.linear_fp8_block(*out[1], w2, s2)):
            if sync:
                torch.cuda.synchronize()
            out.append(f())
        return out[2], res

    def run(sync):
        seen = []
        for x in xs:
            y, res = x, x
            for _ in range(6):
                y, res = step(y, res, sync)
                seen.append(y)
        torch.cuda.synchronize()
        return seen

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    assert fm.linear_fp8_block_status() == (0, 0)


def test_refusals_on_tensors(ops):
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ops.add_rmsnorm_fp8(x.float(), None, g, 1e-6)
    with pytest.raises(ValueError):
        ops.add_rmsnorm_fp8(x, x[:3], g, 1e-6)
    with pytest.raises(ValueError):
        ops.add_rmsnorm_fp8(x[:, ::2], None, g[:128], 1e-6)
    with pytest.raises(ValueError):
        ops.swiglu_fp8(x[:, :255])
    with pytest.raises(fm.Fp4MoeError) as e:
        ops.swiglu_fp8(x[:, :40])  # I = 20: not a multiple of 16
    assert e.value.code == fm.STATUS_CODE["FP4MOE_ERR_UNSUPPORTED_SHAPE"]
    with pytest.raises(fm.Fp4MoeError) as e:
        ops.add_rmsnorm_fp8(x[:, 1:241], None, g[:240], 1e-6)  # rows start off a 16-byte boundary
    assert e.value.code == fm.STATUS_CODE["FP4MOE_ERR_INVALID_ARG"]
    a = [dev(v) for v in linear_inputs(4, 256, 128, 1)]
    with pytest.raises(ValueError):
        ops.linear_fp8_block(a[0], a[1][:, :1], a[2], a[3])
    with pytest.raises(ValueError):
        ops.linear_fp8_block(a[0], a[1], a[2].t(), a[3])
    with pytest.raises(ValueError):
        ops.linear_fp8_block(*a, out_dtype=torch.float16)
    with pytest.raises(fm.Fp4MoeError) as e:
        ops.linear_fp8_block(*a, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == fm.STATUS_CODE["FP4MOE_ERR_WORKSPACE"]
    empty = ops.linear_fp8_block(a[0][:0], a[1][:0], a[2], a[3])
    assert tuple(empty.shape) == (0, 128)
    assert ops.swiglu_fp8(x[:0])[0].shape == (0, 128) and ops.add_rmsnorm_fp8(x[:0], None, g, 1e-6)[2].shape == (0, 256)
    xq, xs, idx, wts, w, sh = expert_inputs(17, 256, 128, 4, 2, 1)
    with pytest.raises(fm.Fp4MoeError) as e:
        ops.experts_fp8_block(*[dev(v) for v in (xq, xs, idx, wts, *w)])  # more than 16 tokens
    assert e.value.code == fm.STATUS_CODE["FP4MOE_ERR_UNSUPPORTED_SHAPE"]


@pytest.mark.parametrize("T,H,I,E,k", [(1, 4096, 128, 4, 1), (4, 4096, 512, 16, 4), (8, 512, 256, 32, 4)])
def test_experts_calls_in_a_row_on_one_workspace(ops, T, H, I, E, k):
    """Each call starts while the one before it ends and both use one workspace: the same outputs
    as calls that wait (units of a CTA of their own, and shared by clusters)."""
    import torch
    xq, xs, idx, wts, w, _ = expert_inputs(T, H, I, E, k, 21)
    wd = [dev(v) for v in w]
    calls = [[dev(v) for v in (np.roll(xq, 128 * i, 1), xs, (idx + i) % E, wts + i)] for i in range(6)]
    ws = torch.empty(fm.experts_fp8_block_workspace_size(fm.make_dims(T, H, I, E, k, fmt=fm.FP8)), dtype=torch.uint8,
                     device="cuda")
    want = []
    for a in calls:
        want.append(ops.experts_fp8_block(*a, *wd, ws=ws))
        torch.cuda.synchronize()
    got = [torch.empty_like(v) for v in want]
    for _ in range(20):
        for a, o in zip(calls, got):
            ops.experts_fp8_block(*a, *wd, out=o, ws=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
