"""One layer object on two streams, and the block-scaled FP8 operators in a
captured graph."""
import numpy as np
import pytest

import block_scaled_fp4_sigmoid_gb300 as fm

from gpu_util import ensure_built, torch_cuda
from test_gpu_fp8_block import bf16, dev, expert_inputs, linear_inputs

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


@pytest.mark.parametrize("T,K,N", [(1024, 1024, 7168), (8, 1040, 8001), (140, 2704, 300)])
def test_products_in_a_captured_graph(ops, T, K, N):
    """Two launches a call, a weight stream and clusters, two calls in a row on one output."""
    import torch
    a, b = [[dev(v) for v in linear_inputs(T, K, N, seed)] for seed in (51, 52)]
    want = [ops.linear_fp8_block(*v) for v in (a, b)]
    got = [torch.zeros_like(want[0]) for _ in want]
    out = torch.zeros_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for v, o in zip((a, b), got):
            ops.linear_fp8_block(*v, out=out)
            o.copy_(out)
    for _ in range(3):
        for o in (out, *got):
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(got, want))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 4096, 128, 4, 1), (7, 512, 1024, 24, 6), (16, 512, 256, 48, 8)])
def test_experts_in_a_captured_graph(ops, T, H, I, E, k):
    """Gate/up units and output columns shared by clusters, and neither."""
    import torch
    xq, xs, idx, wts, w, sh = expert_inputs(T, H, I, E, k, 53, shared=True)
    a = [dev(v) for v in (xq, xs, idx, wts, *w, *sh)]
    want = ops.experts_fp8_block(*a)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.experts_fp8_block(*a, out=out)
        twice = out.clone()
        ops.experts_fp8_block(*a, out=out)
    for _ in range(3):
        out.zero_()
        twice.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(twice, want)


def test_a_layer_in_a_captured_graph(ops):
    """Scratch and outputs of a captured call belong to the graph."""
    import torch
    T, H, I, E, k = 4, 512, 256, 16, 4
    w, sh = [[dev(v) for v in part] for part in expert_inputs(T, H, I, E, k, 54, shared=True)[4:]]
    rng = np.random.default_rng(55)
    gamma, wr = bf16(np.ones(H))[0], bf16(rng.standard_normal((E, H)) * 0.05)[0]
    dims = fm.make_dims(T, H, I, E, k, n_shared=1, routed_scaling=2.5, fmt=fm.FP8)
    layer = ops.Fp8BlockMoE(dims, gamma, wr, dev((0.1 * rng.standard_normal(E)).astype(np.float32)), *w, *sh)
    x = bf16(rng.standard_normal((T, H)))[0]
    other = bf16(rng.standard_normal((T, H)))[0]
    want = [layer.forward(v, v)[0] for v in (x, other)]
    held = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = layer.forward(held, held)
    for v, w0 in zip((other, x), reversed(want)):
        held.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w0)
