"""Workloads of the block-scaled FP8 operators: the fused residual + RMS norm
with E4M3 output, the SwiGLU with E4M3 output, the block-scaled FP8 linear and
the few-token FP8 experts.

Activations hold one fp32 scale per token and 128 columns, weights one per
128 x 128 block.  ``own`` chooses between plain fp32 tensor algebra and the
library's kernels; both take what ``prepare`` returns.
"""
import math

import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # one decode step's input norm: launch latency
        {"name": "norm_token", "op": "norm", "T": 1, "H": 7168, "residual": True, "y": True},
        # an odd batch over a short hidden size with a last block of 80, no residual
        {"name": "norm_ragged", "op": "norm", "T": 333, "H": 2000, "residual": False, "y": False},
        # the norm before the router and the experts of a prefill step
        {"name": "norm_prefill", "op": "norm", "T": 4096, "H": 7168, "residual": True, "y": True},
        # the shared expert's activation in a decode step
        {"name": "swiglu_decode", "op": "swiglu", "T": 8, "I": 2048},
        # the activation of a wide dense layer in prefill
        {"name": "swiglu_prefill", "op": "swiglu", "T": 4096, "I": 18432},
        # a narrow projection of one token: latency, N ends inside a scale block
        {"name": "linear_token", "op": "linear", "T": 1, "K": 7168, "N": 2112, "fp32": False},
        # the gate/up product of a wide dense layer in a decode step: weight stream
        {"name": "linear_decode", "op": "linear", "T": 8, "K": 7168, "N": 36864, "fp32": False},
        # the shared expert's down product of an odd mixed batch, fp32 output
        {"name": "linear_mixed", "op": "linear", "T": 177, "K": 2048, "N": 7168, "fp32": True},
        # the shared expert's gate/up product in prefill
        {"name": "linear_prefill", "op": "linear", "T": 4096, "K": 7168, "N": 4096, "fp32": False},
        # a square projection of the 16k-token batch: tensor bound
        {"name": "linear_large", "op": "linear", "T": 16384, "K": 7168, "N": 7168, "fp32": False},
        # one token through 8 of 256 experts and the shared one
        {"name": "experts_token", "op": "experts", "T": 1, "H": 7168, "I": 2048, "E": 256, "k": 8, "ranks": 1,
         "shared": True},
        # a decode batch over 384 experts
        {"name": "experts_decode", "op": "experts", "T": 8, "H": 7168, "I": 2048, "E": 384, "k": 8, "ranks": 1,
         "shared": False},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], uniform over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "linear", "linear", "linear", "experts"])
    while True:
        if op == "norm":
            c = {"op": op, "T": _spread(rng, 1, 16384), "H": _spread(rng, 256, 16384, 16),
                 "residual": rng.random() < 0.7, "y": rng.random() < 0.5}
        elif op == "swiglu":
            c = {"op": op, "T": _spread(rng, 1, 16384), "I": _spread(rng, 128, 18432, 16)}
        elif op == "linear":
            c = {"op": op, "T": _spread(rng, 1, 16384), "K": _spread(rng, 256, 18432, rng.choice([16, 128])),
                 "N": _spread(rng, 64, 36864, rng.choice([1, 64])), "fp32": rng.random() < 0.2}
        else:
            E = _spread(rng, 8, 384)
            c = {"op": op, "T": _spread(rng, 1, 16), "H": _spread(rng, 256, 7168, 256),
                 "I": _spread(rng, 128, 2048, 128), "E": E, "k": rng.randint(1, min(8, E)),
                 "ranks": rng.choice([1, 1, 4]), "shared": rng.random() < 0.5}
        if 3072 in c.values():
            continue
        w = work(c)
        if op in ("norm", "swiglu") and w["bytes"] > 800e6:
            continue
        if op == "linear" and (w["flops"] > 1.6e12 or w["bytes"] > 800e6):
            continue
        return c


def _blocks(n):
    return -(-n // BLOCK)


def _touched(c):
    """Expected number of distinct experts that T tokens touch on this rank."""
    return c["E"] * (1 - (1 - c["k"] / (c["E"] * c["ranks"])) ** c["T"])


def work(c):
    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        per = 2 + 1 + (4 if c["residual"] else 0) + (2 if c["y"] else 0)
        return {"bytes": T * (H * per + 4 * _blocks(H)) + 2 * H, "flops": 8 * T * H}
    if c["op"] == "swiglu":
        return {"bytes": T * (5 * c["I"] + 4 * _blocks(c["I"])), "flops": 10 * T * c["I"]}
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        return {"bytes": (T + N) * K + 4 * _blocks(K) * (T + _blocks(N)) + T * N * (4 if c["fp32"] else 2),
                "flops": 2 * T * K * N}
    H, I = c["H"], c["I"]
    n = _touched(c) + (1 if c["shared"] else 0)
    routes = T * (c["k"] / c["ranks"] + (1 if c["shared"] else 0))
    return {"bytes": n * 3 * H * I * (1 + 4 / BLOCK ** 2) + T * (H + 4 * _blocks(H)) + 8 * T * c["k"] + 2 * T * H,
            "flops": 6 * routes * H * I}


# --------------------------------------------------------------------- inputs
def _normal_codes(g, *shape):
    """E4M3 codes of normal values, scaled as a block whose largest value is near 448 is (bytes)."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        v = torch.randn(part.numel(), generator=g, device="cuda").mul_(110).clamp_(-448, 448)
        part.copy_(v.to(E4M3).view(torch.uint8))
    return out


def _scales(g, level, *shape):
    return torch.rand(shape, generator=g, device="cuda").add_(0.5).mul_(level)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T = c["T"]
    rows = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    empty = lambda dtype, *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        H = c["H"]
        return {"case": c, "x": rows(T, H).bfloat16(), "residual": rows(T, H).mul_(2).bfloat16() if c["residual"] else None,
                "gamma": rows(H).mul_(0.1).add_(1).bfloat16(),
                "residual_out": empty(torch.bfloat16, T, H) if c["residual"] else None,
                "y": empty(torch.bfloat16, T, H) if c["y"] else None,
                "q": empty(torch.uint8, T, H), "s": empty(torch.float32, T, _blocks(H))}
    if c["op"] == "swiglu":
        I = c["I"]
        return {"case": c, "gu": rows(T, 2 * I).bfloat16(), "q": empty(torch.uint8, T, I),
                "s": empty(torch.float32, T, _blocks(I))}
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        return {"case": c, "xq": _normal_codes(g, T, K), "xs": _scales(g, 0.01, T, _blocks(K)),
                "w": _normal_codes(g, N, K), "ws": _scales(g, 0.0002, _blocks(N), _blocks(K)),
                "out": empty(torch.float32 if c["fp32"] else torch.bfloat16, T, N)}
    H, I, E, k = c["H"], c["I"], c["E"], c["k"]
    idx = torch.rand((T, E * c["ranks"]), generator=g, device="cuda").argsort(dim=1)[:, :k]
    wts = torch.rand((T, k), generator=g, device="cuda") + 0.1
    s = {"case": c, "xq": _normal_codes(g, T, H), "xs": _scales(g, 0.01, T, _blocks(H)),
         "idx": torch.where(idx < E, idx, -1).to(torch.int32),  # -1: an expert that another rank holds
         "wts": wts / wts.sum(1, keepdim=True) * 2.5,
         "w13": _normal_codes(g, E, 2 * I, H), "s13": _scales(g, 0.0002, E, 2 * I // BLOCK, H // BLOCK),
         "w2": _normal_codes(g, E, H, I), "s2": _scales(g, 0.0002, E, H // BLOCK, I // BLOCK),
         "sh13": None, "ss13": None, "sh2": None, "ss2": None, "out": empty(torch.bfloat16, T, H)}
    if c["shared"]:
        s |= {"sh13": _normal_codes(g, 2 * I, H), "ss13": _scales(g, 0.0002, 2 * I // BLOCK, H // BLOCK),
              "sh2": _normal_codes(g, H, I), "ss2": _scales(g, 0.0002, H // BLOCK, I // BLOCK)}
    return s


# ----------------------------------------------------------------- plain form
def _quantize(v):
    """E4M3 codes and fp32 scales of rows v [.., n] in blocks of 128 columns."""
    n = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    s = b.abs().amax(-1) / 448
    q = torch.where(s[..., None] > 0, b / s[..., None], b * 0)
    return q.flatten(-2)[..., :n].to(E4M3), s


def _rows(q, s):
    """fp32 values of codes [.., n] with one scale per 128 columns."""
    return q.view(E4M3).float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _tiles(q, s):
    """fp32 values of codes [.., m, n] with one scale per 128 x 128 block."""
    return _rows(q, s.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :])


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_norm(s):
    z = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    y = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    q, sc = _quantize(y)
    return {"residual": z.bfloat16() if s["residual"] is not None else None,
            "y": y.bfloat16() if s["y"] is not None else None, "q": q, "s": sc}


def _plain_mlp(x, w13, s13, w2, s2):
    """[n, r, H] rows through n experts' gate/up, requantised SwiGLU and down products."""
    gu = x @ _tiles(w13, s13).transpose(-1, -2)
    I = gu.shape[-1] // 2
    hq, hs = _quantize(_silu(gu[..., :I]) * gu[..., I:])
    return _rows(hq, hs) @ _tiles(w2, s2).transpose(-1, -2)


def _plain_experts(s):
    T, k = s["idx"].shape
    x = _rows(s["xq"], s["xs"])
    e = s["idx"].long().clamp(min=0).flatten()
    y = _plain_mlp(x.repeat_interleave(k, 0)[:, None], s["w13"][e], s["s13"][e], s["w2"][e], s["s2"][e])
    wts = torch.where(s["idx"] >= 0, s["wts"], 0)
    out = (y.view(T, k, -1) * wts[..., None]).sum(1)
    if s["sh13"] is not None:
        out = out + _plain_mlp(x, s["sh13"], s["ss13"], s["sh2"], s["ss2"])
    return out.bfloat16()


def run(s):
    op = s["case"]["op"]
    if own:
        from block_scaled_fp4_sigmoid_gb300 import fp8_block as f
        if op == "norm":
            f.add_rmsnorm_fp8(s["x"], s["residual"], s["gamma"], EPS, residual_out=s["residual_out"], y=s["y"],
                              q=s["q"], scales=s["s"])
            return {"residual": s["residual_out"], "y": s["y"], "q": s["q"].view(E4M3), "s": s["s"]}
        if op == "swiglu":
            f.swiglu_fp8(s["gu"], q=s["q"], scales=s["s"])
            return {"q": s["q"].view(E4M3), "s": s["s"]}
        if op == "linear":
            return f.linear_fp8_block(s["xq"], s["xs"], s["w"], s["ws"], out=s["out"])
        return f.experts_fp8_block(s["xq"], s["xs"], s["idx"], s["wts"], s["w13"], s["s13"], s["w2"], s["s2"],
                                   s["sh13"], s["ss13"], s["sh2"], s["ss2"], out=s["out"])
    if op == "norm":
        return _plain_norm(s)
    if op == "swiglu":
        I = s["case"]["I"]
        gu = s["gu"].float()
        q, sc = _quantize(_silu(gu[:, :I]) * gu[:, I:])
        return {"q": q, "s": sc}
    if op == "linear":
        return (_rows(s["xq"], s["xs"]) @ _tiles(s["w"], s["ws"]).T).to(s["out"].dtype)
    return _plain_experts(s)


# ---------------------------------------------------------------------- exact
def _e4m3_round(v):
    """Nearest E4M3 value (ties to even) of float64 v, |v| <= 448."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 1
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def _col(s, n):
    return s.double().repeat_interleave(BLOCK, -1)[..., :n]


def _wvalue(q, s):
    m, n = q.shape
    return q.view(E4M3).to(torch.float64) * _col(s, n).repeat_interleave(BLOCK, 0)[:m]


def _block_amax(v):
    n = v.shape[-1]
    return torch.stack([v[..., i:i + BLOCK].abs().amax(-1) for i in range(0, n, BLOCK)], -1)


def _exact_quantized(v):
    """Unrounded codes (values over scales) and scales in 64 bits."""
    s = _block_amax(v) / 448
    return v / _col(s, v.shape[-1]).clamp(min=1e-300), s


def _exact_mlp(x, w13, s13, w2, s2):
    gu = _wvalue(w13, s13) @ x
    I = gu.shape[0] // 2
    q, s = _exact_quantized((gu[:I] * torch.sigmoid(gu[:I]) * gu[I:])[None])
    return _wvalue(w2, s2) @ (_e4m3_round(q) * _col(s, I))[0]


def exact(c, seed):
    """The results in 64 bits; 8-bit outputs as the values before their rounding."""
    s = prepare(c, seed)
    if c["op"] == "norm":
        z = s["x"].double()
        if s["residual"] is not None:
            z = z + s["residual"].double()
        y = z / torch.sqrt((z * z).sum(-1, keepdim=True) / c["H"] + EPS) * s["gamma"].double()
        q, sc = _exact_quantized(y)
        return {"residual": z if s["residual"] is not None else None, "y": y if s["y"] is not None else None, "q": q,
                "s": sc}
    if c["op"] == "swiglu":
        gate, up = s["gu"].double().chunk(2, -1)
        q, sc = _exact_quantized(gate * torch.sigmoid(gate) * up)
        return {"q": q, "s": sc}
    if c["op"] == "linear":
        K = c["K"]
        out = torch.empty((c["T"], c["N"]), dtype=torch.float64, device="cuda")
        x = s["xq"].view(E4M3).to(torch.float64) * _col(s["xs"], K)
        for n in range(0, c["N"], 4096):
            q = s["w"][n:n + 4096]
            out[:, n:n + 4096] = x @ _wvalue(q, s["ws"][n // BLOCK:n // BLOCK + 4096 // BLOCK]).T
        return out
    T, H = c["T"], c["H"]
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for t in range(T):
        x = s["xq"][t].view(E4M3).to(torch.float64) * _col(s["xs"][t], H)
        for j in range(c["k"]):
            e = int(s["idx"][t, j])
            if e >= 0:
                out[t] += float(s["wts"][t, j]) * _exact_mlp(x, s["w13"][e], s["s13"][e], s["w2"][e], s["s2"][e])
        if c["shared"]:
            out[t] += _exact_mlp(x, s["sh13"], s["ss13"], s["sh2"], s["ss2"])
    return out
