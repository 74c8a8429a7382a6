"""Host-side checks of the block-scaled FP8 entry points: sizes and arguments
that are refused before any device work, and the workspace sizes.  No compute
entry point gets past its argument checks here."""
import ctypes

import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
from block_scaled_fp4_sigmoid_gb300 import build

OK, INVALID, SHAPE, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return fm.lib()


P = 1 << 20  # an aligned address that no call dereferences


def norm(lib, **kw):
    a = dict(x=P, x_ld=256, residual=None, gamma=P, T=4, H=256, eps=1e-6, residual_out=None, y=None, q=P, scales=P)
    a.update(kw)
    return lib.fp4moe_add_rmsnorm_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(gamma=None), INVALID), (dict(q=None, scales=None), INVALID),
    (dict(scales=None), INVALID), (dict(q=None), INVALID), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=264), SHAPE),
    (dict(H=65552), SHAPE), (dict(x_ld=248), INVALID), (dict(x_ld=260), INVALID), (dict(x=P + 2), INVALID),
    (dict(y=P + 8), INVALID), (dict(scales=P + 2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(T=0), OK), (dict(T=0, q=None, scales=None, y=P), OK)])
def test_norm_arguments(lib, kw, code):
    assert norm(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(gu=None), INVALID), (dict(q=None), INVALID), (dict(T=-2), SHAPE), (dict(I=24), SHAPE), (dict(gu_ld=500), INVALID),
    (dict(gu_ld=516), INVALID), (dict(gu=P + 4), INVALID), (dict(q=P + 8), INVALID), (dict(T=0), OK)])
def test_swiglu_arguments(lib, kw, code):
    a = dict(gu=P, gu_ld=512, T=4, I=256, q=P, scales=P)
    a.update(kw)
    assert lib.fp4moe_swiglu_fp8(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(xq=None), INVALID), (dict(ws=None), WORKSPACE), (dict(out=None), INVALID), (dict(K=24), SHAPE), (dict(K=0), SHAPE),
    (dict(N=0), SHAPE), (dict(T=-1), SHAPE), (dict(ws_bytes=16), WORKSPACE), (dict(out_ld=127), INVALID),
    (dict(xq=P + 8), INVALID), (dict(w=P + 1), INVALID), (dict(out=P + 1), INVALID),
    (dict(out=P + 2, out_is_fp32=1), INVALID), (dict(T=0), OK), (dict(T=0, ws=None, ws_bytes=0), OK)])
def test_linear_arguments(lib, kw, code):
    a = dict(T=4, K=256, N=128, xq=P, xs=P, w=P, w_scale=P, out=P, out_ld=128, out_is_fp32=0, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    assert lib.fp4moe_linear_fp8_block(*a.values(), None) == code


def test_linear_workspace(lib):
    assert lib.fp4moe_linear_fp8_block_workspace_size(4, 20, 128) == 0
    assert lib.fp4moe_linear_fp8_block_workspace_size(-1, 256, 128) == 0
    for T, K, N in ((0, 256, 1), (1, 16, 1), (4096, 7168, 36864), (1 << 20, 65536, 1 << 20)):
        assert fm.linear_fp8_block_workspace_size(T, K, N) >= 256


def experts(lib, dims, w, **kw):
    a = dict(xq=P, xs=P, idx=P, wts=P, out=P, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return lib.fp4moe_experts_fp8_block(ctypes.byref(dims), ctypes.byref(w), *a.values(), None)


def test_experts_arguments_and_workspace(lib):
    d = fm.make_dims(16, 256, 128, 8, 2, fmt=fm.FP8)
    full = fm.Fp8BlockWeights(*[P] * 8)
    assert experts(lib, d, full, xq=None) == INVALID
    assert experts(lib, d, full, xq=P + 8) == INVALID
    assert experts(lib, d, full, idx=P + 2) == INVALID
    assert experts(lib, d, full, ws_bytes=64) == WORKSPACE
    assert experts(lib, d, fm.Fp8BlockWeights(P, P, None, P)) == INVALID
    assert experts(lib, fm.make_dims(16, 256, 128, 8, 2, fmt=fm.MXFP4), full) == INVALID
    assert experts(lib, fm.make_dims(17, 256, 128, 8, 2, fmt=fm.FP8), full) == SHAPE
    assert experts(lib, fm.make_dims(16, 320, 128, 8, 2, fmt=fm.FP8), full) == SHAPE
    shared = fm.make_dims(16, 256, 128, 8, 2, n_shared=1, fmt=fm.FP8)
    assert experts(lib, shared, fm.Fp8BlockWeights(P, P, P, P)) == INVALID
    # the requantised h of every route (and of the shared expert) fits, in rows of eight tokens
    for T, E, k, sh in ((1, 8, 1, 0), (16, 8, 2, 1), (16, 512, 16, 1), (16, 16, 16, 0)):
        n = fm.experts_fp8_block_workspace_size(fm.make_dims(T, 256, 128, E, k, n_shared=sh, fmt=fm.FP8))
        entries = T * k if E >= T * k else max(E, -(-T * k // 8))
        assert n >= 8 * (entries + sh * -(-T // 8)) * (128 + 4)
    assert lib.fp4moe_experts_fp8_block_workspace_size(ctypes.byref(fm.make_dims(17, 256, 128, 8, 2, fmt=fm.FP8))) == 0
