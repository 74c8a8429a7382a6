"""The few-token experts at sizes that a rank of an expert-parallel layer meets
and hidden sizes of an odd number of scale blocks, against the FP64 oracle with
the tolerance of the other expert tests: 2^-16 of the magnitudes, the bf16
rounding, and how far rounding h to E4M3 can move the output."""
import numpy as np
import pytest

from oracle import fp8_block as B

from gpu_util import ensure_built, torch_cuda
from test_gpu_fp8_block import U_BF16, dev, expert_inputs, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    torch_cuda()
    ensure_built()
    from block_scaled_fp4_sigmoid_gb300 import fp8_block
    return fp8_block


@pytest.mark.parametrize("T,H,I,E,k,shared", [(1, 256, 128, 6, 8, False), (8, 512, 256, 6, 8, True), (16, 512, 128, 3, 16, True),
                                              (13, 384, 256, 1, 16, False), (3, 128, 128, 4, 2, True),
                                              (16, 640, 384, 24, 6, False), (1, 4224, 128, 2, 4, False)])
def test_fewer_experts_than_a_token_chooses_and_odd_hidden_sizes(ops, T, H, I, E, k, shared):
    import torch
    xq, xs, _, wts, w, sh = expert_inputs(T, H, I, E, 1, 41, shared=shared)
    rng = np.random.default_rng(42)
    # each token's k routes over 64 experts, of which this rank holds the first E
    idx = np.argsort(rng.random((T, 64)), axis=1)[:, :k].astype(np.int32)
    idx[0, :2] = [-1, E - 1]
    idx = np.where(idx < E, idx, -1).astype(np.int32)
    wts = (0.1 + rng.random((T, k))).astype(np.float32)
    ref, S, A = B.experts(xq, xs, idx, wts, *w, shared=sh or None)
    a = [dev(v) for v in (xq, xs, idx, wts, *w, *sh)]
    got = ops.experts_fp8_block(*a)
    bad = np.abs(f64(got) - ref) > U_BF16 * (np.abs(ref) + A) + B.ACC * S + A
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    assert torch.equal(got, ops.experts_fp8_block(*a))


def test_every_route_on_one_expert(ops):
    """Sixteen routes a token, all to the rank's one expert: their weights add."""
    T, H, I, k = 16, 256, 128, 16
    xq, xs, _, _, w, _ = expert_inputs(T, H, I, 1, 1, 43)
    idx, wts = np.zeros((T, k), np.int32), np.full((T, k), 1 / 16, np.float32)
    ref, S, A = B.experts(xq, xs, idx, wts, *w)
    got = f64(ops.experts_fp8_block(*[dev(v) for v in (xq, xs, idx, wts, *w)]))
    assert np.all(np.abs(got - ref) <= U_BF16 * (np.abs(ref) + A) + B.ACC * S + A)
