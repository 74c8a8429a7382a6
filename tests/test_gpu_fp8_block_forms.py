"""Every form of the block-scaled FP8 linear against the FP64 oracle, at shapes
that are asserted (test_fp8_block_forms_cpu.py) to select it: the output within
2^-16 of the sum of the terms' magnitudes and one rounding to its type."""
import numpy as np
import pytest

import test_gpu_fp8_block as base
from oracle import fp8_block as B
from test_fp8_block_forms_cpu import CHAINS, FORMS

from gpu_util import ensure_built, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    torch_cuda()
    ensure_built()
    from block_scaled_fp4_sigmoid_gb300 import fp8_block
    return fp8_block


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,K,N", [s for v in FORMS.values() for s in v])
def test_form(ops, T, K, N, fp32):
    """The product, written into columns of a wider output that start off 16 bytes; nothing else is
    written, and a second call gives the same bits."""
    import torch
    inputs = base.linear_inputs(T, K, N, T + K + N)
    y, S = B.linear(*inputs)
    a = [base.dev(v) for v in inputs]
    wide = torch.full((T + 2, N + 7), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    got = ops.linear_fp8_block(*a, out=wide[1:T + 1, 3:N + 3])
    bad = np.abs(base.f64(got) - y) > (base.U_F32 if fp32 else base.U_BF16) * np.abs(y) + B.ACC * S
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    assert torch.equal(ops.linear_fp8_block(*a, out_dtype=wide.dtype), got)
    got.fill_(7.0)
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("T,K,N", [v[0] for v in FORMS.values() if v[0][0] > 1 and v[0][1] > 128])
def test_nan_stays_in_its_row_and_column(ops, T, K, N):
    xq, xs, wq, ws = base.linear_inputs(T, K, N, 6)
    t, n = T - 1, N - 2
    xq[t, 130] = 0x7F
    wq[n, K - 1] = 0xFF
    got = base.f64(ops.linear_fp8_block(*[base.dev(v) for v in (xq, xs, wq, ws)]))
    assert np.all(np.isnan(got[t])) and np.all(np.isnan(got[:, n]))
    assert np.isfinite(np.delete(np.delete(got, t, 0), n, 1)).all()


@pytest.mark.parametrize("T,H,I", CHAINS)
def test_calls_in_a_row(ops, T, H, I):
    """The streamed forms that fetch weights before the launch before them has ended."""
    base.test_calls_in_a_row_equal_calls_that_wait(ops, T, H, I)
