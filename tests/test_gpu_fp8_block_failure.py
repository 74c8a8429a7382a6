"""A device wait of the block-scaled FP8 linear that runs out, without a fault:
CTA 0 withholds its first pipeline stage under a limit of 1 ms on the waits.
The call must record FP4MOE_ERR_TIMEOUT (in the workspace, or without one in
the library's word), drain what it issued, meet its cluster and return; the
next normal call on the same stream is correct and its status clear.  Each
tensor-core form is covered: whole tiles of either width, two launches, and
clusters of two, four and eight."""
import numpy as np
import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
import test_gpu_fp8_block as base
from oracle import fp8_block as B
from test_fp8_block_forms_cpu import FORMS

from gpu_util import ensure_built, torch_cuda

pytestmark = pytest.mark.gpu

TIMEOUT = fm.STATUS_CODE["FP4MOE_ERR_TIMEOUT"]


@pytest.fixture(scope="module")
def ops():
    torch_cuda()
    ensure_built()
    from block_scaled_fp4_sigmoid_gb300 import fp8_block
    return fp8_block


def debug(withhold):
    d = fm.Debug()
    d.wait_limit_ns = 1_000_000
    d.withhold_first_stage = withhold
    return d


@pytest.mark.parametrize("own_word", [True, False])
@pytest.mark.parametrize("T,K,N", [v[0] for f, v in FORMS.items() if f.startswith("tensor")])
def test_withheld_stage_times_out_and_recovers(ops, T, K, N, own_word):
    import torch
    inputs = base.linear_inputs(T, K, N, 61)
    y, S = B.linear(*inputs)
    a = [base.dev(v) for v in inputs]
    want = ops.linear_fp8_block(*a)
    out = torch.empty_like(want)
    ws = torch.full((256,), 0xA5, dtype=torch.uint8, device="cuda") if own_word else None
    status = (lambda: fm.get_status(ws.data_ptr(), s)) if own_word else (lambda: fm.linear_fp8_block_status(s))
    s = torch.cuda.current_stream().cuda_stream
    fm.linear_fp8_block_status(s)

    def call(withhold):
        fm.linear_fp8_block_debug(T, K, N, *[v.data_ptr() for v in a], out.data_ptr(), N, False, debug(withhold),
                                  ws.data_ptr() if own_word else None, 256 if own_word else 0, s)
        torch.cuda.synchronize()  # the call returned and the stream drained: no fault, no hang

    call(1)
    st, n = status()
    assert st == TIMEOUT and n >= 1, (st, n)
    # the limit alone lets an ordinary call through; it clears the workspace's word (the library's was read)
    out.fill_(7.0)
    call(0)
    assert status() == (0, 0)
    assert torch.equal(out, want)
    got = ops.linear_fp8_block(*a, out=out.fill_(7.0), ws=ws)
    assert np.all(np.abs(base.f64(got) - y) <= base.U_BF16 * np.abs(y) + B.ACC * S)
    assert status() == (0, 0)


def test_the_streamed_forms_wait_for_nothing(ops):
    import torch
    T, K, N = FORMS["stream 1x2x4"][1]
    a = [base.dev(v) for v in base.linear_inputs(T, K, N, 62)]
    want = ops.linear_fp8_block(*a)
    out = torch.empty_like(want)
    s = torch.cuda.current_stream().cuda_stream
    fm.linear_fp8_block_debug(T, K, N, *[v.data_ptr() for v in a], out.data_ptr(), N, False, debug(1), None, 0, s)
    assert torch.equal(out, want)
    assert fm.linear_fp8_block_status(s) == (0, 0)
