// Block-scaled FP8 activations: residual addition + RMS norm, and SwiGLU,
// each with E4M3 codes and one fp32 scale per 128 columns.
//
// Both read their inputs once and write their outputs once (HBM bound; the
// norm up to 16384 columns): a thread loads 8 consecutive columns at a time (16
// bytes of bf16), 16 or 8 lanes share a scale block, whose largest magnitude is a
// shuffle reduction.
#include <algorithm>

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4moe {

namespace {

struct NormParams {
  const uint16_t *x, *residual, *gamma;
  uint16_t *residual_out, *y;
  uint8_t* q;
  float* scales;
  int64_t x_ld;
  int T, H;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
}

// Codes of 8 values over a scale s with reciprocal r.
__device__ __forceinline__ void store_codes(const float* v, float s, float r, uint8_t* q) {
  float t[8];
  if (s >= 1.17549435e-38f) {  // (one test for the eight)
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = v[j] * r;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = e4m3_scaled(v[j], s, r);
  }
  *reinterpret_cast<uint2*>(q) = make_uint2(e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7]));
}

// Codes and scale of the 16-lane group's block from each lane's 8 values; all
// 16 lanes take part (v = 0 past the row's end).
__device__ __forceinline__ void quant_block(const float* v, bool in, uint8_t* q, float* scale) {
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[j]));
#pragma unroll
  for (int o = 8; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffu << (threadIdx.x & 16), amax, o));
  const float s = e4m3_scale(amax);
  if (in) {
    store_codes(v, s, __fdiv_rn(1.f, s), q);
    if ((threadIdx.x & 15) == 0) *scale = s;
  }
}

// A CTA takes rows blockIdx.x, + gridDim.x, ...; CH 8-column chunks of a row
// per thread, kept in registers between the sum of squares and the output.
// Up to two chunks the next row's inputs are fetched before this row's
// reduction and stores, so that reads never pause: 4096 x 7168 with residual
// and y in 42 us (6.3 TB/s) against 47 us with a CTA per row.  (With more
// chunks they would not fit the registers.)  Longer rows are right but not
// fast: from 16400 columns on the 64 registers of a thread of 1024 do not hold its
// part of the row (2048 x 16384 52 us, 5.8 TB/s; 2048 x 16400 83 us, 3.6; 512 x
// 65536 175 us, 1.7).
template <int CH>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormParams p) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_trigger();
  const int chunks = p.H >> 3, nb = blocks128(p.H), warps = (int)(blockDim.x >> 5);
  uint4 xw[CH], rw[CH];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      xw[i] = make_uint4(0, 0, 0, 0);
      if (c < chunks) {
        xw[i] = *reinterpret_cast<const uint4*>(p.x + row * p.x_ld + 8 * c);
        if (p.residual) rw[i] = *reinterpret_cast<const uint4*>(p.residual + row * p.H + 8 * c);
      }
    }
  };
  fetch(blockIdx.x);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, buf ^= 1) {
    float v[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      unpack8(xw[i], v[i]);
      if (c < chunks) {
        if (p.residual) {
          float r[8];
          unpack8(rw[i], r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        }
        if (p.residual_out) *reinterpret_cast<uint4*>(p.residual_out + row * p.H + 8 * c) = pack8(v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    if (CH <= 2 && row + gridDim.x < p.T) fetch(row + gridDim.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) part[buf][threadIdx.x >> 5] = ss;
    __syncthreads();  // (the other buffer is written next: no second barrier)
    ss = 0.f;
    for (int w = 0; w < warps; ++w) ss += part[buf][w];
    const float r = rsqrtf(__fdiv_rn(ss, (float)p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = i * blockDim.x + threadIdx.x;
      const bool in = c < chunks;
      if (in) {
        float g[8];
        unpack8(*reinterpret_cast<const uint4*>(p.gamma + 8 * c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * g[j];
        if (p.y) *reinterpret_cast<uint4*>(p.y + row * p.H + 8 * c) = pack8(v[i]);
      }
      if (p.q) quant_block(v[i], in, p.q + row * p.H + 8 * c, p.scales + row * nb + (c >> 4));
    }
    if (CH > 2 && row + gridDim.x < p.T) fetch(row + gridDim.x);
  }
}

// Eight lanes a scale block: lane l takes columns 8 l .. and 64 + 8 l .. of it.
// Blocks are blockDim.x threads along a row by blockDim.y rows, so that no
// index is divided.  Issue slots ran out before the memory did (81% of them at
// 4096 x 18432 with 16 lanes of 8 columns, 67 us; with a flat index, divided
// by the row's length, 69 us), so the block's reduction and its two divisions
// are shared by 16 columns a lane.
__global__ void __launch_bounds__(256) swiglu_fp8_kernel(const uint16_t* gu, int64_t gu_ld, int T, int I, uint8_t* q,
                                                         float* scales) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int l = threadIdx.x & 7, b = blockIdx.y * (blockDim.x >> 3) + (threadIdx.x >> 3), nb = blocks128(I);
  if (row >= T || b >= nb) return;  // whole groups of lanes
  const int c0 = b * kBlk + 8 * l;
  const uint16_t* src = gu + row * gu_ld + c0;
  float h[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint4 gw = make_uint4(0, 0, 0, 0), uw = gw;
    if (c0 + 64 * k < I) gw = ldg_stream(src + 64 * k), uw = ldg_stream(src + I + 64 * k);
    float g[8], u[8];
    unpack8(gw, g);
    unpack8(uw, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[k][j] = swiglu(g[j], u[j]);
  }
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) amax = max_nan(amax, fabsf(h[j >> 3][j & 7]));
  const uint32_t lanes = 0xffu << ((threadIdx.y * blockDim.x + threadIdx.x) & 24);
#pragma unroll
  for (int o = 4; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(lanes, amax, o));
  const float s = e4m3_scale(amax), r = __fdiv_rn(1.f, s);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (c0 + 64 * k < I) store_codes(h[k], s, r, q + row * I + c0 + 64 * k);
  if (l == 0) scales[row * nb + b] = s;
}

}  // namespace

cudaError_t launch_add_rmsnorm(const uint16_t* x, int64_t x_ld, const uint16_t* residual, const uint16_t* gamma, int T,
                               int H, float eps, uint16_t* residual_out, uint16_t* y, uint8_t* q, float* scales,
                               cudaStream_t s) {
  const NormParams p{x, residual, gamma, residual_out, y, q, scales, x_ld, T, H, eps};
  const int chunks = H / 8;
  int ch = 1;  // at most 512 threads, up to 1024 from 8192 columns on
  while (ch < 8 && chunks > (ch == 1 ? 512 : 1024) * ch) ch *= 2;
  const int threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
  // as many CTAs as fit an SM's registers with the prefetch (1792 threads)
  const dim3 block((unsigned)threads), grid((unsigned)std::min(T, 152 * std::max(1, 1792 / threads)));
  switch (ch) {
    case 1: return launch_pdl(add_rmsnorm_kernel<1>, grid, block, 0, s, p);
    case 2: return launch_pdl(add_rmsnorm_kernel<2>, grid, block, 0, s, p);
    case 4: return launch_pdl(add_rmsnorm_kernel<4>, grid, block, 0, s, p);
    default: return launch_pdl(add_rmsnorm_kernel<8>, grid, block, 0, s, p);
  }
}

cudaError_t launch_swiglu_fp8(const uint16_t* gu, int64_t gu_ld, int T, int I, uint8_t* q, float* scales,
                              cudaStream_t s) {
  const int nb = blocks128(I), bx = 8 * std::min(nb, 32), by = 256 / bx;
  const dim3 grid((unsigned)((T + by - 1) / by), (unsigned)((8 * nb + bx - 1) / bx));
  return launch_pdl(swiglu_fp8_kernel, grid, dim3(bx, by), 0, s, gu, gu_ld, T, I, q, scales);
}

}  // namespace fp4moe

using namespace fp4moe;

namespace {
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
constexpr int32_t kMaxRows = 1 << 20;  // rows of one call
constexpr int32_t kMaxCols = 65536;
bool experts_sizes_ok(const fp4moe_dims& d) {
  return d.T >= 0 && d.T <= kExpertsMaxT && d.H >= kBlk && d.H <= kMaxCols && d.H % kBlk == 0 && d.I >= kBlk &&
         d.I <= kMaxCols && d.I % kBlk == 0 && d.E >= 1 && d.E <= kExpertsMaxE && d.top_k >= 1 &&
         d.top_k <= kExpertsMaxK && (d.n_shared == 0 || d.n_shared == 1);
}
}  // namespace

extern "C" {

fp4moe_status fp4moe_add_rmsnorm_fp8(const uint16_t* x, int64_t x_ld, const uint16_t* residual, const uint16_t* gamma,
                                     int32_t T, int32_t H, float eps, uint16_t* residual_out, uint16_t* y, uint8_t* q,
                                     float* scales, void* stream) {
  if (!x || !gamma || (!y && !q) || (q != nullptr) != (scales != nullptr)) return FP4MOE_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxRows || H < 16 || H > kMaxCols || H % 16 != 0) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (x_ld < H || x_ld % 8 != 0 || !(eps >= 0.f)) return FP4MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(q, 16) || !aligned(scales, 4))
    return FP4MOE_ERR_INVALID_ARG;
  if (T == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  return cuda_status(
      launch_add_rmsnorm(x, x_ld, residual, gamma, T, H, eps, residual_out, y, q, scales, static_cast<cudaStream_t>(stream)));
}

fp4moe_status fp4moe_swiglu_fp8(const uint16_t* gu, int64_t gu_ld, int32_t T, int32_t I, uint8_t* q, float* scales,
                                void* stream) {
  if (!gu || !q || !scales) return FP4MOE_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxRows || I < 16 || I > kMaxCols || I % 16 != 0) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (gu_ld < 2 * (int64_t)I || gu_ld % 8 != 0) return FP4MOE_ERR_INVALID_ARG;
  if (!aligned(gu, 16) || !aligned(q, 16) || !aligned(scales, 4)) return FP4MOE_ERR_INVALID_ARG;
  if (T == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  return cuda_status(launch_swiglu_fp8(gu, gu_ld, T, I, q, scales, static_cast<cudaStream_t>(stream)));
}

size_t fp4moe_linear_fp8_block_workspace_size(int32_t T, int32_t K, int32_t N) {
  if (T < 0 || T > kMaxRows || K < 16 || K > kMaxCols || K % 16 != 0 || N < 1 || N > kMaxRows) return 0;
  return linear_fp8_workspace(T, K, N);
}

const char* fp4moe_linear_fp8_block_form(int32_t T, int32_t K, int32_t N) {
  return fp4moe_linear_fp8_block_workspace_size(T, K, N) == 0 ? "unsupported" : T == 0 ? "none" : linear_fp8_form(T, K, N);
}

fp4moe_status fp4moe_linear_fp8_block(int32_t T, int32_t K, int32_t N, const uint8_t* xq, const float* xs,
                                      const uint8_t* w, const float* w_scale, void* out, int64_t out_ld,
                                      int32_t out_is_fp32, void* ws, size_t ws_bytes, void* stream) {
  return fp4moe_linear_fp8_block_debug(T, K, N, xq, xs, w, w_scale, out, out_ld, out_is_fp32, nullptr, ws, ws_bytes,
                                       stream);
}

fp4moe_status fp4moe_linear_fp8_block_debug(int32_t T, int32_t K, int32_t N, const uint8_t* xq, const float* xs,
                                            const uint8_t* w, const float* w_scale, void* out, int64_t out_ld,
                                            int32_t out_is_fp32, const fp4moe_debug* dbg, void* ws, size_t ws_bytes,
                                            void* stream) {
  if (!xq || !xs || !w || !w_scale || !out) return FP4MOE_ERR_INVALID_ARG;
  const size_t need = fp4moe_linear_fp8_block_workspace_size(T, K, N);
  if (need == 0) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (ws ? ws_bytes < need : ws_bytes != 0) return FP4MOE_ERR_WORKSPACE;
  if (out_ld < N || !aligned(xq, 16) || !aligned(w, 16) || !aligned(xs, 4) || !aligned(w_scale, 4) ||
      !aligned(out, out_is_fp32 ? 4 : 2) || !aligned(ws, 16))
    return FP4MOE_ERR_INVALID_ARG;
  if (T == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  const LinearFp8Args a{T, K, N, xq, xs, w, w_scale, out, out_ld, out_is_fp32 != 0, ws,
                        dbg && dbg->wait_limit_ns > 0 ? (uint64_t)dbg->wait_limit_ns : 0,
                        dbg && dbg->withhold_first_stage != 0};
  return cuda_status(launch_linear_fp8(a, static_cast<cudaStream_t>(stream)));
}

fp4moe_status fp4moe_linear_fp8_block_status(void* stream, fp4moe_status* st, int64_t* count) {
  if (fp4moe_status e = check_device()) return e;
  int32_t* word = nullptr;
  if (linear_fp8_status_word(&word) != cudaSuccess) return FP4MOE_ERR_CUDA;
  const fp4moe_status e = fp4moe_get_status(word, stream, st, count);
  return e ? e : fp4moe_clear_status(word, stream);
}

size_t fp4moe_experts_fp8_block_workspace_size(const fp4moe_dims* dims) {
  if (!dims || dims->fmt != FP4MOE_FP8 || !experts_sizes_ok(*dims)) return 0;
  return experts_fp8_workspace(*dims);
}

fp4moe_status fp4moe_experts_fp8_block(const fp4moe_dims* dims, const fp4moe_fp8_block_weights* w, const uint8_t* xq,
                                       const float* xs, const int32_t* topk_idx, const float* topk_w, uint16_t* out,
                                       void* ws, size_t ws_bytes, void* stream) {
  if (!dims || !w || !xq || !xs || !topk_idx || !topk_w || !out || !ws) return FP4MOE_ERR_INVALID_ARG;
  if (dims->fmt != FP4MOE_FP8) return FP4MOE_ERR_INVALID_ARG;
  const size_t need = fp4moe_experts_fp8_block_workspace_size(dims);
  if (need == 0) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < need) return FP4MOE_ERR_WORKSPACE;
  if (!w->w13 || !w->w13_scale || !w->w2 || !w->w2_scale) return FP4MOE_ERR_INVALID_ARG;
  if (dims->n_shared && (!w->sh13 || !w->sh13_scale || !w->sh2 || !w->sh2_scale)) return FP4MOE_ERR_INVALID_ARG;
  for (const void* q : {(const void*)xq, (const void*)w->w13, (const void*)w->w2, (const void*)w->sh13,
                        (const void*)w->sh2, (const void*)out, (const void*)ws})
    if (!aligned(q, 16)) return FP4MOE_ERR_INVALID_ARG;
  for (const void* q : {(const void*)xs, (const void*)w->w13_scale, (const void*)w->w2_scale,
                        (const void*)w->sh13_scale, (const void*)w->sh2_scale, (const void*)topk_idx,
                        (const void*)topk_w})
    if (!aligned(q, 4)) return FP4MOE_ERR_INVALID_ARG;
  if (dims->T == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  return cuda_status(
      launch_experts_fp8(*dims, *w, xq, xs, topk_idx, topk_w, out, ws, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
