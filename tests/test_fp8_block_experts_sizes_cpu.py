"""Sizes that the few-token experts take, host side: what the call itself needs,
not the routing limits of the whole layer."""
import ctypes

import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
from block_scaled_fp4_sigmoid_gb300 import build

INVALID, SHAPE = 1, 2
P = 1 << 20  # an aligned address that no call dereferences


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return fm.lib()


def call(lib, d, **kw):
    """The code of a call that is refused at the latest for its workspace of 0 bytes (3)."""
    a = dict(xq=P, xs=P, idx=P, wts=P, out=P, ws=P, ws_bytes=0)
    a.update(kw)
    w = fm.Fp8BlockWeights(*[P] * 8)
    return lib.fp4moe_experts_fp8_block(ctypes.byref(d), ctypes.byref(w), *a.values(), None)


def dims(**kw):
    a = dict(T=4, H=256, I=128, E=8, top_k=2, fmt=fm.FP8)
    a.update(kw)
    return fm.make_dims(**a)


TAKEN = [
    dict(E=6, top_k=8), dict(E=1, top_k=16),     # a rank that holds fewer experts than a token chooses
    dict(E=6, n_group=4, topk_group=1),          # routing parameters, which are not used
    dict(E=12, n_group=0, topk_group=9), dict(routed_scaling=float("nan")),
    dict(H=384), dict(H=128), dict(T=1), dict(T=16), dict(E=512, top_k=16), dict(I=65536), dict(H=65536),
]


@pytest.mark.parametrize("kw", TAKEN, ids=str)
def test_sizes_that_the_kernels_take(lib, kw):
    d = dims(**kw)
    entries = min(d.E, d.T * d.top_k)
    assert lib.fp4moe_experts_fp8_block_workspace_size(ctypes.byref(d)) >= entries * 8 * (d.I + d.I // 128 * 4)
    assert call(lib, d) == 3  # only the workspace is too small


@pytest.mark.parametrize("kw", [dict(T=17), dict(T=-1), dict(H=64), dict(H=320), dict(H=65664), dict(I=64), dict(I=200),
                                dict(I=65664), dict(E=0), dict(E=513), dict(top_k=0), dict(top_k=17), dict(n_shared=2),
                                dict(n_shared=-1)], ids=str)
def test_sizes_that_they_do_not_take(lib, kw):
    d = dims(**kw)
    assert lib.fp4moe_experts_fp8_block_workspace_size(ctypes.byref(d)) == 0
    assert call(lib, d, ws_bytes=1 << 40) == SHAPE


def test_a_call_without_tokens_does_nothing(lib):
    d = dims(T=0)
    n = fm.experts_fp8_block_workspace_size(d)
    assert n > 0
    assert call(lib, d, ws_bytes=n) == 0
    assert call(lib, d, xq=None) == INVALID


def test_the_tensor_function_without_tokens():
    """A batch that is empty on this rank: an empty output, nothing launched (there is no device here)."""
    torch = pytest.importorskip("torch")
    from block_scaled_fp4_sigmoid_gb300 import fp8_block as fb
    E, H, I = 4, 256, 128
    with pytest.MonkeyPatch.context() as m:
        m.setattr(fb, "_device", lambda t: t.get_device())
        m.setattr(fb, "_current_device", lambda: -1)
        m.setattr(fb, "_experts", lambda *a: pytest.fail("launched"))
        u8, f32 = lambda *s: torch.zeros(s, dtype=torch.uint8), lambda *s: torch.zeros(s)  # noqa: E731
        out = torch.zeros((0, H), dtype=torch.bfloat16)
        got = fb.experts_fp8_block(u8(0, H), f32(0, 2), torch.zeros((0, 2), dtype=torch.int32), f32(0, 2), u8(E, 2 * I, H),
                                   f32(E, 2, 2), u8(E, H, I), f32(E, 2, 1), out=out)
    assert got is out
