// Block-scaled FP8 experts for few tokens, in two kernels: gate/up + SwiGLU +
// E4M3 requantisation, then down + weighted combine.
//
// Every column of the MMAs is a token (8 NT columns for up to 16 tokens), so
// an expert's weights are read once for all its tokens, and both kernels only
// visit experts that some token chose.
#include <algorithm>

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4moe {

namespace {

constexpr int kMaxE = 512, kMaxTok = kExpertsMaxT, kMaxRoutes = 16 * kMaxTok;
constexpr int kMaxList = kMaxRoutes + 1;  // chosen experts and the shared one

struct ExpertsParams {
  const uint8_t *xq, *w13, *w2, *sh13, *sh2;
  const float *xs, *s13, *s2, *ss13, *ss2;
  const int32_t* idx;
  const float* wts;
  uint8_t* hq;   // [list position * T + token, I]
  float* hs;     // [list position * T + token, I / 128]
  uint16_t* out;
  int T, H, I, E, k, shared;
};

struct ExpertList {
  uint32_t mask[kMaxE + 1];  // tokens that chose the expert
  uint16_t e[kMaxList];      // chosen experts, ascending; the shared one is E
  int n;
};

// Lists the chosen experts; both kernels of a call get the same list.  Routes
// outside [0, E) (an expert that another rank holds) choose nothing.
__device__ __forceinline__ void list_experts(const ExpertsParams& p, ExpertList& L) {
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) L.mask[e] = 0u;
  __syncthreads();
  for (int r = threadIdx.x; r < p.T * p.k; r += blockDim.x) {
    const int e = p.idx[r];
    if (e >= 0 && e < p.E) atomicOr(&L.mask[e], 1u << (r / p.k));
  }
  if (threadIdx.x == 0 && p.shared) L.mask[p.E] = (1u << p.T) - 1u;
  __syncthreads();
  if (threadIdx.x < 32) {
    int n = 0;
    for (int e0 = 0; e0 <= p.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const bool on = e <= p.E && L.mask[e] != 0u;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      if (on) L.e[n + __popc(m & ((1u << threadIdx.x) - 1u))] = (uint16_t)e;
      n += __popc(m);
    }
    if (threadIdx.x == 0) L.n = n;
  }
  __syncthreads();
}

constexpr int kGuThreads = 512;

// One unit: 128 gate and 128 up rows (one scale block of h) of one expert.
// Warp = 16 gate rows and the 16 up rows of the same h values, over every
// second K block.
template <int NT>
__global__ void __launch_bounds__(kGuThreads) experts_gateup_kernel(const ExpertsParams p) {
  __shared__ ExpertList L;
  __shared__ float part[8][8 * NT][32];
  __shared__ float amax[8][8 * NT];
  __shared__ __align__(16) uint8_t codes[8 * NT][128];  // read as 16-byte words
  pdl_wait();
  pdl_trigger();
  list_experts(p, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rg = warp & 7, kh = warp >> 3;
  const int hb = p.H / kBlk, ib = p.I / kBlk, units = L.n * ib;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int u = unit / ib, b = unit - u * ib, e = L.e[u];
    const uint32_t mask = L.mask[e];
    const bool sh = e == p.E;
    const uint8_t* w = sh ? p.sh13 : p.w13 + (int64_t)e * 2 * p.I * p.H;
    const float* ws = sh ? p.ss13 : p.s13 + (int64_t)e * 2 * ib * hb;
    const uint8_t* row = w + (int64_t)(b * kBlk + 16 * rg + g) * p.H;
    const float *wsg = ws + (int64_t)b * hb, *wsu = ws + (int64_t)(ib + b) * hb;
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
    for (int kb = kh; kb < hb; kb += 2) {
      uint4 wv[2][4], x[2];
      const int64_t k0 = kb * kBlk + 16 * t;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          wv[m][j] = ldg_stream(row + (int64_t)(m * p.I + 8 * (j >> 1)) * p.H + k0 + 64 * (j & 1));
      const float sg = wsg[kb], su = wsu[kb];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint8_t* xr = p.xq + (int64_t)min(8 * i + g, p.T - 1) * p.H + k0;
        x[0] = *reinterpret_cast<const uint4*>(xr);
        x[1] = *reinterpret_cast<const uint4*>(xr + 64);
        const float x0 = p.xs[min(8 * i + 2 * t, p.T - 1) * hb + kb];
        const float x1 = p.xs[min(8 * i + 2 * t + 1, p.T - 1) * hb + kb];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_block(d, wv[m], x);
          const float sw = m ? su : sg, s0 = sw * x0, s1 = sw * x1;
          acc[m][i][0] = fmaf(s0, d[0], acc[m][i][0]);
          acc[m][i][1] = fmaf(s1, d[1], acc[m][i][1]);
          acc[m][i][2] = fmaf(s0, d[2], acc[m][i][2]);
          acc[m][i][3] = fmaf(s1, d[3], acc[m][i][3]);
        }
      }
    }
    // the odd K blocks' sums join the even ones'
    if (kh) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[rg][(m * NT + i) * 4 + j][lane] = acc[m][i][j];
    }
    __syncthreads();
    float h[NT][4];
    if (!kh) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[i][j] = swiglu(acc[0][i][j] + part[rg][i * 4 + j][lane], acc[1][i][j] + part[rg][(NT + i) * 4 + j][lane]);
        // columns 2t (j = 0, 2) and 2t + 1: largest |h| over the warp's 16 rows
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a = max_nan(fabsf(h[i][c]), fabsf(h[i][c + 2]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
          if (g == 0) amax[rg][8 * i + 2 * t + c] = a;
        }
      }
    }
    __syncthreads();
    if (!kh) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int tok = 8 * i + 2 * t + c;
          float a = amax[0][tok];
#pragma unroll
          for (int q = 1; q < 8; ++q) a = max_nan(a, amax[q][tok]);
          const float s = e4m3_scale(a);
          const float r = __fdiv_rn(1.f, s);
          const uint32_t two = e4m3x4(e4m3_scaled(h[i][c], s, r), e4m3_scaled(h[i][c + 2], s, r), 0.f, 0.f);
          codes[tok][16 * rg + g] = (uint8_t)two;
          codes[tok][16 * rg + g + 8] = (uint8_t)(two >> 8);
          if (rg == 0 && g == 0 && ((mask >> tok) & 1u)) p.hs[(int64_t)(u * p.T + tok) * ib + b] = s;
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 8 * NT * 8; o += kGuThreads) {
      const int tok = o >> 3, c = 16 * (o & 7);
      if ((mask >> tok) & 1u)
        *reinterpret_cast<uint4*>(p.hq + (int64_t)(u * p.T + tok) * p.I + b * kBlk + c) =
            *reinterpret_cast<const uint4*>(&codes[tok][c]);
    }
  }
}

constexpr int kDnWarps = 8;

// One CTA: 16 output columns (rows of every chosen expert's W2), all tokens.
// The (expert, K block) pairs go to the warps in turn; each adds weight *
// scales * product into its token columns, and the warps' sums are joined in
// warp order, so the result does not depend on timing.
template <int NT>
__global__ void __launch_bounds__(32 * kDnWarps) experts_down_kernel(const ExpertsParams p) {
  __shared__ ExpertList L;
  __shared__ float rw[kMaxList][8 * NT];  // routing weight of (list position, token)
  __shared__ float part[kDnWarps][NT * 4][32];
  pdl_wait();
  pdl_trigger();
  list_experts(p, L);
  for (int o = threadIdx.x; o < L.n * 8 * NT; o += blockDim.x) {
    const int u = o / (8 * NT), tok = o - u * 8 * NT, e = L.e[u];
    float v = 0.f;
    if (tok < p.T) {
      if (e == p.E)
        v = 1.f;
      else
        for (int j = 0; j < p.k; ++j)
          if (p.idx[tok * p.k + j] == e) v += p.wts[tok * p.k + j];
    }
    rw[u][tok] = v;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16, hb = p.H / kBlk, ib = p.I / kBlk, items = L.n * ib;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int it = warp; it < items; it += kDnWarps) {
    const int u = it / ib, b = it - u * ib, e = L.e[u];
    const uint32_t mask = L.mask[e];
    const bool sh = e == p.E;
    const uint8_t* w = (sh ? p.sh2 : p.w2 + (int64_t)e * p.H * p.I) + (int64_t)(n0 + g) * p.I + b * kBlk + 16 * t;
    const float sw = (sh ? p.ss2 : p.s2 + (int64_t)e * hb * ib)[(n0 / kBlk) * ib + b];
    uint4 wv[4], x[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) wv[j] = ldg_stream(w + (int64_t)8 * (j >> 1) * p.I + 64 * (j & 1));
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int tok = 8 * i + g, c0 = 8 * i + 2 * t, c1 = c0 + 1;
      // a token that did not choose the expert has no h: its column is zero
      // and takes nothing (not even a NaN of the weights)
      x[0] = x[1] = make_uint4(0, 0, 0, 0);
      if ((mask >> tok) & 1u) {
        const uint8_t* h = p.hq + (int64_t)(u * p.T + tok) * p.I + b * kBlk + 16 * t;
        x[0] = *reinterpret_cast<const uint4*>(h);
        x[1] = *reinterpret_cast<const uint4*>(h + 64);
      }
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_block(d, wv, x);
      if ((mask >> c0) & 1u) {
        const float s = rw[u][c0] * (sw * p.hs[(int64_t)(u * p.T + c0) * ib + b]);
        acc[i][0] = fmaf(s, d[0], acc[i][0]);
        acc[i][2] = fmaf(s, d[2], acc[i][2]);
      }
      if ((mask >> c1) & 1u) {
        const float s = rw[u][c1] * (sw * p.hs[(int64_t)(u * p.T + c1) * ib + b]);
        acc[i][1] = fmaf(s, d[1], acc[i][1]);
        acc[i][3] = fmaf(s, d[3], acc[i][3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][4 * i + j][lane] = acc[i][j];
  __syncthreads();
  for (int o = threadIdx.x; o < 128 * NT; o += 32 * kDnWarps) {
    const int tok = o >> 4, r = o & 15, i = tok >> 3, c = tok & 7;
    const int l = 4 * (r & 7) + (c >> 1), j = 4 * i + 2 * (r >> 3) + (c & 1);
    float v = 0.f;
#pragma unroll
    for (int wq = 0; wq < kDnWarps; ++wq) v += part[wq][j][l];
    if (tok < p.T) p.out[(int64_t)tok * p.H + n0 + r] = f32_to_bf16_rn(v);
  }
}

int64_t list_cap(const fp4moe_dims& d) { return std::min(d.E, d.T * d.top_k) + d.n_shared; }

int64_t hq_bytes(const fp4moe_dims& d) { return (list_cap(d) * d.T * d.I + 255) / 256 * 256; }

template <int NT>
cudaError_t launch(const ExpertsParams& p, int64_t cap, int sms, cudaStream_t s) {
  const int64_t units = cap * (p.I / kBlk);
  cudaError_t e = launch_pdl(experts_gateup_kernel<NT>, dim3((unsigned)std::min<int64_t>(units, 2 * sms)),
                             dim3(kGuThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(experts_down_kernel<NT>, dim3(p.H / 16), dim3(32 * kDnWarps), 0, s, p);
  return e;
}

}  // namespace

size_t experts_fp8_workspace(const fp4moe_dims& d) {
  return (size_t)(hq_bytes(d) + list_cap(d) * d.T * (d.I / kBlk) * 4);
}

cudaError_t launch_experts_fp8(const fp4moe_dims& d, const fp4moe_fp8_block_weights& w, const uint8_t* xq,
                               const float* xs, const int32_t* topk_idx, const float* topk_w, uint16_t* out, void* ws,
                               cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  ExpertsParams p;
  p.xq = xq, p.xs = xs, p.idx = topk_idx, p.wts = topk_w, p.out = out;
  p.w13 = w.w13, p.s13 = w.w13_scale, p.w2 = w.w2, p.s2 = w.w2_scale;
  p.sh13 = w.sh13, p.ss13 = w.sh13_scale, p.sh2 = w.sh2, p.ss2 = w.sh2_scale;
  p.hq = static_cast<uint8_t*>(ws);
  p.hs = reinterpret_cast<float*>(p.hq + hq_bytes(d));
  p.T = d.T, p.H = d.H, p.I = d.I, p.E = d.E, p.k = d.top_k, p.shared = d.n_shared;
  return d.T <= 8 ? launch<1>(p, list_cap(d), sms, s) : launch<2>(p, list_cap(d), sms, s);
}

}  // namespace fp4moe
