// Block-scaled FP8 linear: out[t, n] = sum_b xs[t, b] ws[n / 128, b] *
// sum_{k in block b} xq[t, k] w[n, k], E4M3 values, fp32 sums, bf16 or fp32 out.
#include <algorithm>

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4moe {

namespace {

struct StreamParams {
  const uint8_t *xq, *w;
  const float *xs, *ws;
  void* out;
  int64_t out_ld;
  int32_t* status;  // cleared here; this kernel waits for nothing
  int T, K, N, out_fp32;
};

constexpr int kStreamWarps = 8;

// Few tokens: a CTA owns 16 weight rows and 8 NT tokens; its warps take the
// 128-column blocks in turn, each streaming weights straight from global
// memory into mma.sync operands, and their sums are joined in warp order.
template <int NT>
__global__ void __launch_bounds__(32 * kStreamWarps) linear_stream_kernel(const StreamParams p) {
  __shared__ float part[kStreamWarps][NT * 4][32];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kStatusInts) p.status[threadIdx.x] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * (8 * NT), nb = blocks128(p.K);
  const float* ws = p.ws + (int64_t)(n0 / kBlk) * nb;
  const uint8_t* wrow[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) wrow[i] = p.w + (int64_t)min(n0 + g + 8 * i, p.N - 1) * p.K;  // past N: not stored
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int b = warp; b < nb; b += kStreamWarps) {
    uint4 w[4], x[2];
    const int k0 = b * kBlk + 16 * t;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = k0 + 64 * j < p.K;
      w[j] = in ? ldg_stream(wrow[0] + k0 + 64 * j) : zero;
      w[2 + j] = in ? ldg_stream(wrow[1] + k0 + 64 * j) : zero;
    }
    const float sw = ws[b];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* xr = p.xq + (int64_t)min(t0 + 8 * i + g, p.T - 1) * p.K + k0;
#pragma unroll
      for (int j = 0; j < 2; ++j) x[j] = k0 + 64 * j < p.K ? *reinterpret_cast<const uint4*>(xr + 64 * j) : zero;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_block(d, w, x);
      const float s0 = sw * p.xs[(int64_t)min(t0 + 8 * i + 2 * t, p.T - 1) * nb + b];
      const float s1 = sw * p.xs[(int64_t)min(t0 + 8 * i + 2 * t + 1, p.T - 1) * nb + b];
      acc[i][0] = fmaf(s0, d[0], acc[i][0]);
      acc[i][1] = fmaf(s1, d[1], acc[i][1]);
      acc[i][2] = fmaf(s0, d[2], acc[i][2]);
      acc[i][3] = fmaf(s1, d[3], acc[i][3]);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][4 * i + j][lane] = acc[i][j];
  __syncthreads();
  // thread -> (token, row): 16 consecutive rows of one token are adjacent
  for (int o = threadIdx.x; o < 128 * NT; o += 32 * kStreamWarps) {
    const int tok = o >> 4, r = o & 15, i = tok >> 3, c = tok & 7;
    const int l = 4 * (r & 7) + (c >> 1), j = 4 * i + 2 * (r >> 3) + (c & 1);
    float v = 0.f;
#pragma unroll
    for (int wq = 0; wq < kStreamWarps; ++wq) v += part[wq][j][l];
    if (t0 + tok < p.T && n0 + r < p.N) {
      const int64_t at = (int64_t)(t0 + tok) * p.out_ld + n0 + r;
      if (p.out_fp32)
        static_cast<float*>(p.out)[at] = v;
      else
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rn(v);
    }
  }
}

}  // namespace

size_t linear_fp8_workspace(int, int, int) { return 256; }

cudaError_t launch_linear_fp8(const LinearFp8Args& a, cudaStream_t s) {
  const StreamParams p{a.xq, a.w, a.xs, a.ws, a.out, a.out_ld, static_cast<int32_t*>(a.scratch), a.T, a.K, a.N, a.out_fp32 ? 1 : 0};
  const unsigned rows = (unsigned)((a.N + 15) / 16);
  // the token tiles are the grid's y dimension: at most 65,535 of them
  const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
  for (int64_t t0 = 0; t0 < a.T; t0 += (int64_t)65535 * 8 * nt) {
    StreamParams q = p;
    q.T = (int)std::min<int64_t>(a.T - t0, (int64_t)65535 * 8 * nt);
    q.xq += t0 * a.K;
    q.xs += t0 * blocks128(a.K);
    q.out = static_cast<uint8_t*>(a.out) + t0 * a.out_ld * (a.out_fp32 ? 4 : 2);
    const dim3 grid(rows, (unsigned)((q.T + 8 * nt - 1) / (8 * nt))), block(32 * kStreamWarps);
    const cudaError_t e = nt == 1   ? launch_pdl(linear_stream_kernel<1>, grid, block, 0, s, q)
                          : nt == 2 ? launch_pdl(linear_stream_kernel<2>, grid, block, 0, s, q)
                                    : launch_pdl(linear_stream_kernel<4>, grid, block, 0, s, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fp4moe
