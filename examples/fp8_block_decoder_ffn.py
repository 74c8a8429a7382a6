"""The feed-forward sublayers of a decoder on block-scaled FP8 weights, one decode
step and one prompt: norm -> router -> experts, and norm -> gate/up -> SwiGLU ->
down, with random weights.

    python examples/fp8_block_decoder_ffn.py [--tokens 8] [--prompt 512] [--hidden 1024] [--inter 512] [--experts 32]

Prints the time of each sublayer call and how far its output is from the same
sublayer in fp32 on the dequantised weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_sigmoid_gb300 as fm  # noqa: E402
from block_scaled_fp4_sigmoid_gb300 import fp8_block as fb  # noqa: E402


def random_weight(*shape):
    """(E4M3 codes, fp32 scales per 128 x 128 block) of N(0, 0.02) weights."""
    w = torch.randn(shape, device="cuda") * 0.02
    m, n = shape[-2:]
    b = w.unflatten(-1, (n // 128, 128)).unflatten(-3, (m // 128, 128))
    s = b.abs().amax((-1, -3)) / 448
    q = (b / s[..., :, None, :, None]).flatten(-2).flatten(-3, -2).to(torch.float8_e4m3fn)
    return q, s.contiguous()


def value(q, s):
    return q.float() * s.repeat_interleave(128, -2).repeat_interleave(128, -1)


def ms(fn, n=20):
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def norm(x, res, gamma, eps=1e-6):
    z = x.float() + res.float()
    return z * torch.rsqrt(z.square().mean(-1, keepdim=True) + eps) * gamma.float()


def mlp(x, w13, w2):
    g, u = (x @ w13.T).chunk(2, -1)
    return (torch.nn.functional.silu(g) * u) @ w2.T


def main():
    p = argparse.ArgumentParser()
    for name, default in (("tokens", 8), ("prompt", 512), ("hidden", 1024), ("inter", 512), ("experts", 32), ("top-k", 4)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    torch.manual_seed(0)
    H, I, E, T = a.hidden, a.inter, a.experts, a.tokens
    w13, s13 = random_weight(E, 2 * I, H)
    w2, s2 = random_weight(E, H, I)
    sh13, ss13 = random_weight(2 * I, H)
    sh2, ss2 = random_weight(H, I)
    gamma = (1 + 0.1 * torch.randn(H, device="cuda")).bfloat16()
    wr = (torch.randn(E, H, device="cuda") * 0.02).bfloat16()
    bias = 0.1 * torch.randn(E, device="cuda")

    dims = fm.make_dims(T, H, I, E, a.top_k, n_shared=1, routed_scaling=2.5, fmt=fm.FP8)
    moe = fb.Fp8BlockMoE(dims, gamma, wr, bias, w13, s13, w2, s2, sh13, ss13, sh2, ss2)
    x, res = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
    out, _ = moe.forward(x, res)
    v = norm(x, res, gamma)
    idx, wts = moe.route(v.bfloat16())
    ref = mlp(v, value(sh13, ss13), value(sh2, ss2))
    for t in range(T):
        for j in range(a.top_k):
            e = int(idx[t, j])
            ref[t] += wts[t, j] * mlp(v[t], value(w13[e], s13[e]), value(w2[e], s2[e]))
    far = float((out.float() - ref).norm() / ref.norm())
    print(f"experts sublayer, {T} tokens: {1e3 * ms(lambda: moe.forward(x, res)):.1f} us, {far:.3f} from fp32")

    dense = fb.Fp8BlockMlp(gamma, sh13, ss13, sh2, ss2)
    for T in (a.tokens, a.prompt):
        x, res = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
        out, _ = dense.forward(x, res)
        ref = mlp(norm(x, res, gamma), value(sh13, ss13), value(sh2, ss2))
        far = float((out.float() - ref).norm() / ref.norm())
        print(f"dense sublayer, {T} tokens: {1e3 * ms(lambda: dense.forward(x, res)):.1f} us, {far:.3f} from fp32")
    status, n = fm.linear_fp8_block_status(torch.cuda.current_stream().cuda_stream)
    if status:
        raise RuntimeError(f"device status {fm.STATUS.get(status, status)} ({n})")


if __name__ == "__main__":
    main()
