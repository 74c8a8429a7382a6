"""One layer object on two streams, and the block-scaled FP8 operators in a
captured graph."""
import numpy as np
import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
from oracle import fp8_block as B

from gpu_util import ensure_built, torch_cuda
from test_gpu_fp8_block import bf16, codes, dev, expert_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    torch_cuda()
    ensure_built()
    from block_scaled_fp4_sigmoid_gb300 import fp8_block
    return fp8_block


@pytest.mark.parametrize("T,H,I,E,k", [(3, 512, 256, 16, 4), (16, 2048, 512, 64, 8)])
def test_one_layer_on_two_streams_equals_calls_that_wait(ops, T, H, I, E, k):
    import torch
    w, sh = [[dev(v) for v in part] for part in expert_inputs(T, H, I, E, k, 31, shared=True)[4:]]
    rng = np.random.default_rng(32)
    gamma, wr = bf16(np.ones(H))[0], bf16(rng.standard_normal((E, H)) * 0.05)[0]
    dims = fm.make_dims(T, H, I, E, k, n_shared=1, routed_scaling=2.5, fmt=fm.FP8)
    layer = ops.Fp8BlockMoE(dims, gamma, wr, dev((0.1 * rng.standard_normal(E)).astype(np.float32)), *w, *sh)
    xs = [bf16(rng.standard_normal((T, H)))[0] for _ in range(2)]
    want = []
    for x in xs:
        want.append(layer.forward(x, x)[0])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(30):
        for s, x, g in zip(streams, xs, got):
            with torch.cuda.stream(s):
                g.append(layer.forward(x, x)[0])
    torch.cuda.synchronize()
    for g, w0 in zip(got, want):
        assert all(torch.equal(v, w0) for v in g)
