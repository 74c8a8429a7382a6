"""Block-scaled FP8 operators on tensors: E4M3 codes with one fp32 scale per
token and 128 columns (activations) or per 128 x 128 block (weights).

The functions check their tensors, allocate what the caller does not pass and
call the library on the current stream of the tensors' device, with that device
current for the call: the library launches on the thread's current device, and
the default stream's handle is the same number on every device.  (Each check is
one expression over all tensors, a few microseconds less than one call a
tensor; what is wrong is worked out only once something is.)  Codes are
torch.uint8 or torch.float8_e4m3fn tensors.  ``Fp8BlockMlp`` and
``Fp8BlockMoE`` run them together as the two feed-forward sublayers of a
decoder layer.
"""
from __future__ import annotations

import torch

from . import (FP8, Dims, Fp8BlockWeights, add_rmsnorm_fp8 as _add_rmsnorm, experts_fp8_block as _experts,
               experts_fp8_block_workspace_size, linear_fp8_block as _linear,
               make_dims, route as _route, swiglu_fp8 as _swiglu, workspace_size)

BLOCK = 128
_CODES = (torch.uint8, torch.float8_e4m3fn)
_bf16, _f32 = torch.bfloat16, torch.float32
_BF16, _F32 = (_bf16,), (_f32,)
_OUT = _BF16 + _F32


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _check(name, t, shape, dtypes, device, dense=True):
    """A tensor of the given shape, one of the types and the device (an index); dense
    (row-major) or, for a matrix, with unit stride along its rows."""
    if t.shape != shape or t.dtype not in dtypes or t.get_device() != device:
        raise ValueError(f"{name}: expected {tuple(shape)} of {dtypes} on cuda:{device}, got {tuple(t.shape)} of {t.dtype} "
                         f"on {t.device}")
    if not (t.is_contiguous() if dense else t.stride(1) == 1 or t.shape[1] <= 1):
        raise ValueError(f"{name}: {'row-major' if dense else 'unit column stride'} expected, strides are {t.stride()}")


def _out(name, t, shape, dtypes, device, dense=True):
    if t is None:
        return torch.empty(shape, dtype=dtypes[0], device=f"cuda:{device}")
    _check(name, t, shape, dtypes, device, dense)
    return t


def _check_ws(ws, device):
    """A workspace: its bytes are all there, on the device."""
    if ws.dtype is not torch.uint8 or ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws: dense uint8 on cuda:{device} expected, got {tuple(ws.shape)} of {ws.dtype} on {ws.device} with "
                         f"strides {ws.stride()}")


def _device(t):
    d = t.get_device()
    if d < 0:
        raise ValueError("CUDA tensors expected")
    return d


# the raw handle of a device's current stream, without a Stream object around it
_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def add_rmsnorm_fp8(x, residual, gamma, eps: float, *, residual_out=None, y=None, q=None, scales=None,
                    want_y: bool = False):
    """z = x + residual, v = z rsqrt(mean(z^2) + eps) gamma; returns (bf16(z), bf16(v), codes of
    v, scales) (fp4moe_add_rmsnorm_fp8).  x bf16 [T, H], rows may be strided; residual bf16
    [T, H] or None (then bf16(z) is x itself).  bf16(v) is written when y is passed or
    want_y is set, else None is returned in its place."""
    if x.dim() != 2:
        raise ValueError(f"x: a matrix expected, got {tuple(x.shape)}")
    shape = x.shape
    T, H = shape
    dev = _device(x)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return add_rmsnorm_fp8(x, residual, gamma, eps, residual_out=residual_out, y=y, q=q, scales=scales, want_y=want_y)
    if residual is not None and residual_out is None:
        residual_out = torch.empty(shape, dtype=_bf16, device=x.device)
    if y is None and want_y:
        y = torch.empty(shape, dtype=_bf16, device=x.device)
    if q is None:
        q = torch.empty(shape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T, (H + 127) // 128), dtype=_f32, device=x.device)
    if not (x.dtype is _bf16 and (x.stride(1) == 1 or H == 1) and gamma.dtype is _bf16 and gamma.shape == (H,)
            and gamma.is_contiguous() and q.dtype in _CODES and q.shape == shape and q.is_contiguous()
            and scales.dtype is _f32 and scales.shape == (T, (H + 127) // 128) and scales.is_contiguous()
            and gamma.get_device() == q.get_device() == scales.get_device() == dev
            and (residual is None or residual.dtype is _bf16 and residual.shape == shape and residual.is_contiguous()
                 and residual.get_device() == dev)
            and (residual_out is None or residual_out.dtype is _bf16 and residual_out.shape == shape
                 and residual_out.is_contiguous() and residual_out.get_device() == dev)
            and (y is None or y.dtype is _bf16 and y.shape == shape and y.is_contiguous() and y.get_device() == dev)):
        _check("x", x, shape, _BF16, dev, dense=False)
        _check("gamma", gamma, (H,), _BF16, dev)
        for name, t in (("residual", residual), ("residual_out", residual_out), ("y", y)):
            if t is not None:
                _check(name, t, shape, _BF16, dev)
        _check("q", q, shape, _CODES, dev)
        _check("scales", scales, (T, _blocks(H)), _F32, dev)
    if T:
        _add_rmsnorm(x.data_ptr(), x.stride(0) if T > 1 else H, None if residual is None else residual.data_ptr(),
                     gamma.data_ptr(), T, H, eps, None if residual_out is None else residual_out.data_ptr(),
                     None if y is None else y.data_ptr(), q.data_ptr(), scales.data_ptr(), _stream(dev))
    return residual_out if residual_out is not None else x, y, q, scales


def swiglu_fp8(gu, *, q=None, scales=None):
    """(codes, scales) of silu(gu[:, :I]) * gu[:, I:] (fp4moe_swiglu_fp8); gu bf16 [T, 2I], rows
    may be strided."""
    if gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError(f"gu: [T, 2I] expected, got {tuple(gu.shape)}")
    T, I = gu.shape
    I //= 2
    dev = _device(gu)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return swiglu_fp8(gu, q=q, scales=scales)
    if q is None:
        q = torch.empty((T, I), dtype=torch.uint8, device=gu.device)
    if scales is None:
        scales = torch.empty((T, (I + 127) // 128), dtype=_f32, device=gu.device)
    if not (gu.dtype is _bf16 and gu.stride(1) == 1 and q.dtype in _CODES and q.shape == (T, I) and q.is_contiguous()
            and scales.dtype is _f32 and scales.shape == (T, (I + 127) // 128) and scales.is_contiguous()
            and q.get_device() == scales.get_device() == dev):
        _check("gu", gu, (T, 2 * I), _BF16, dev, dense=False)
        _check("q", q, (T, I), _CODES, dev)
        _check("scales", scales, (T, _blocks(I)), _F32, dev)
    if T:
        _swiglu(gu.data_ptr(), gu.stride(0) if T > 1 else 2 * I, T, I, q.data_ptr(), scales.data_ptr(), _stream(dev))
    return q, scales


def linear_fp8_block(xq, xs, w, w_scale, *, out=None, out_dtype=torch.bfloat16, ws=None):
    """out [T, N] = x . W^T for codes xq [T, K] with scales xs [T, K/128] and w [N, K] with
    w_scale [N/128, K/128] (fp4moe_linear_fp8_block; blocks rounded up).  out: bf16 or fp32,
    rows may be strided.  ws: None, or a dense uint8 tensor of linear_fp8_block_workspace_size(T, K, N)
    bytes whose status word get_status reads; without it a device-side timeout is recorded in
    the library's word, which linear_fp8_block_status reads."""
    if xq.dim() != 2 or w.dim() != 2:
        raise ValueError(f"xq and w: matrices expected, got {tuple(xq.shape)} and {tuple(w.shape)}")
    (T, K), N = xq.shape, w.shape[0]
    kb = (K + 127) // 128
    dev = _device(xq)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return linear_fp8_block(xq, xs, w, w_scale, out=out, out_dtype=out_dtype, ws=ws)
    if out is None:
        if out_dtype not in _OUT:
            raise ValueError(f"out_dtype: bf16 or fp32, got {out_dtype}")
        out = torch.empty((T, N), dtype=out_dtype, device=xq.device)
    if not (xq.dtype in _CODES and xq.is_contiguous() and xs.dtype is _f32 and xs.shape == (T, kb) and xs.is_contiguous()
            and w.dtype in _CODES and w.shape[1] == K and w.is_contiguous() and w_scale.dtype is _f32
            and w_scale.shape == ((N + 127) // 128, kb) and w_scale.is_contiguous() and out.dtype in _OUT
            and out.shape == (T, N) and (out.stride(1) == 1 or N == 1)
            and xs.get_device() == w.get_device() == w_scale.get_device() == out.get_device() == dev):
        _check("xq", xq, (T, K), _CODES, dev)
        _check("xs", xs, (T, kb), _F32, dev)
        _check("w", w, (N, K), _CODES, dev)
        _check("w_scale", w_scale, (_blocks(N), kb), _F32, dev)
        _check("out", out, (T, N), _OUT, dev, dense=False)
    if ws is not None:
        _check_ws(ws, dev)
    if T:
        _linear(T, K, N, xq.data_ptr(), xs.data_ptr(), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
                out.stride(0) if T > 1 else N, out.dtype is _f32, None if ws is None else ws.data_ptr(),
                0 if ws is None else ws.numel(), _stream(dev))
    elif ws is not None:
        ws.view(-1)[:64].zero_()  # the status word
    return out


def experts_fp8_block(xq, xs, topk_idx, topk_w, w13, w13_scale, w2, w2_scale, sh13=None, sh13_scale=None, sh2=None,
                      sh2_scale=None, *, out=None, ws=None):
    """bf16 [T, H]: the routed experts of up to 16 tokens, plus the shared one where given
    (fp4moe_experts_fp8_block).  xq [T, H], xs [T, H/128]; topk_idx int32 and topk_w fp32 [T, k]
    (an index outside [0, E) is skipped); w13 [E, 2I, H], w2 [E, H, I] with one scale per 128 x
    128 block.  ws: None, or a dense uint8 tensor of experts_fp8_block_workspace_size bytes that no
    call on another stream uses meanwhile."""
    if xq.dim() != 2 or topk_idx.dim() != 2 or w13.dim() != 3:
        raise ValueError(f"xq, topk_idx, w13: two, two and three dimensions expected, got {tuple(xq.shape)}, "
                         f"{tuple(topk_idx.shape)}, {tuple(w13.shape)}")
    (T, H), k, E, I = xq.shape, topk_idx.shape[1], w13.shape[0], w13.shape[1] // 2
    dev = _device(xq)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return experts_fp8_block(xq, xs, topk_idx, topk_w, w13, w13_scale, w2, w2_scale, sh13, sh13_scale, sh2,
                                     sh2_scale, out=out, ws=ws)
    _check("xq", xq, (T, H), _CODES, dev)
    _check("xs", xs, (T, _blocks(H)), _F32, dev)
    _check("topk_idx", topk_idx, (T, k), (torch.int32,), dev)
    _check("topk_w", topk_w, (T, k), _F32, dev)
    hb, ib = _blocks(H), _blocks(I)
    _check("w13", w13, (E, 2 * I, H), _CODES, dev)
    _check("w13_scale", w13_scale, (E, 2 * ib, hb), _F32, dev)
    _check("w2", w2, (E, H, I), _CODES, dev)
    _check("w2_scale", w2_scale, (E, hb, ib), _F32, dev)
    if sh13 is not None:
        _check("sh13", sh13, (2 * I, H), _CODES, dev)
        _check("sh13_scale", sh13_scale, (2 * ib, hb), _F32, dev)
        _check("sh2", sh2, (H, I), _CODES, dev)
        _check("sh2_scale", sh2_scale, (hb, ib), _F32, dev)
    dims = make_dims(T, H, I, E, k, n_shared=int(sh13 is not None), fmt=FP8)
    n = experts_fp8_block_workspace_size(dims)
    out = _out("out", out, (T, H), _BF16, dev)
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device=xq.device)
    else:
        _check_ws(ws, dev)
    if T:
        weights = Fp8BlockWeights(w13.data_ptr(), w13_scale.data_ptr(), w2.data_ptr(), w2_scale.data_ptr(), _ptr(sh13),
                                  _ptr(sh13_scale), _ptr(sh2), _ptr(sh2_scale))
        _experts(dims, weights, xq.data_ptr(), xs.data_ptr(), topk_idx.data_ptr(), topk_w.data_ptr(), out.data_ptr(),
                 ws.data_ptr(), ws.numel(), _stream(dev))
    return out


class Fp8BlockMlp:
    """A dense feed-forward sublayer: norm -> gate/up product -> SwiGLU -> down
    product, on block-scaled FP8 weights w13 [2I, H] (gate rows, then up rows)
    and w2 [H, I]."""

    def __init__(self, gamma, w13, w13_scale, w2, w2_scale, eps: float = 1e-6):
        self.gamma, self.eps = gamma, eps
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13, w13_scale, w2, w2_scale

    def forward(self, x, residual=None):
        """(output bf16 [T, H], residual stream bf16 [T, H]) for x bf16 [T, H]: the caller adds
        the output to the residual stream in its next norm."""
        res, _, q, s = add_rmsnorm_fp8(x, residual, self.gamma, self.eps)
        gu = linear_fp8_block(q, s, self.w13, self.w13_scale)
        hq, hs = swiglu_fp8(gu)
        return linear_fp8_block(hq, hs, self.w2, self.w2_scale), res


class Fp8BlockMoE:
    """A mixture-of-experts feed-forward sublayer for up to 16 tokens: norm ->
    router (fp4moe_route on the bf16 norm output) -> experts (and the shared
    one) on block-scaled FP8 weights.  dims: as make_dims returns for the
    layer with fmt=FP8; w_router bf16 [E, H], bias fp32 [E].  It holds every
    expert that its router chooses from: a rank with some of them calls
    experts_fp8_block itself, with routes of -1 for the others'.  The object keeps
    its weights only: each call's scratch comes from the allocator, so calls on
    several streams do not meet."""

    def __init__(self, dims: Dims, gamma, w_router, bias, w13, w13_scale, w2, w2_scale, sh13=None, sh13_scale=None,
                 sh2=None, sh2_scale=None, eps: float = 1e-6):
        if dims.fmt != FP8 or dims.n_shared != int(sh13 is not None):
            raise ValueError("dims: fmt FP8, and n_shared as the shared expert's weights say")
        self.dims, self.gamma, self.w_router, self.bias, self.eps = dims, gamma, w_router, bias, eps
        self.weights = (w13, w13_scale, w2, w2_scale, sh13, sh13_scale, sh2, sh2_scale)
        self.device = w13.device
        _check("w_router", w_router, (dims.E, dims.H), _BF16, _device(w13))
        _check("bias", bias, (dims.E,), _F32, _device(w13))
        # the router's, then the experts'
        self.ws_bytes = max(workspace_size(dims), experts_fp8_block_workspace_size(dims))

    def _scratch(self):
        return torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)

    def route(self, y, ws=None):
        """(topk_idx, topk_w) of the bf16 rows y [T, H].  ws: None, or a dense uint8 tensor of
        self.ws_bytes bytes."""
        d = self.dims
        dev = _device(self.w_router)
        if _current_device() != dev:
            with torch.cuda.device(dev):
                return self.route(y, ws)
        _check("y", y, (d.T, d.H), _BF16, dev)
        idx = torch.empty((d.T, d.top_k), dtype=torch.int32, device=self.device)
        w = torch.empty((d.T, d.top_k), dtype=torch.float32, device=self.device)
        if ws is None:
            ws = self._scratch()
        else:
            _check_ws(ws, dev)
        _route(d, y.data_ptr(), self.w_router.data_ptr(), self.bias.data_ptr(), idx.data_ptr(), w.data_ptr(), None,
               ws.data_ptr(), ws.numel(), _stream(dev))
        return idx, w

    def forward(self, x, residual=None):
        """As Fp8BlockMlp.forward."""
        res, y, q, s = add_rmsnorm_fp8(x, residual, self.gamma, self.eps, want_y=True)
        ws = self._scratch()
        idx, w = self.route(y, ws)
        return experts_fp8_block(q, s, idx, w, *self.weights, ws=ws), res
