// Block-scaled FP8 linear: out[t, n] = sum_b xs[t, b] ws[n / 128, b] *
// sum_{k in block b} xq[t, k] w[n, k], E4M3 values, fp32 sums, bf16 or fp32 out.

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4moe {

namespace {

struct StreamParams {
  const uint8_t *xq, *w;
  const float *xs, *ws;
  void* out;
  int64_t out_ld;
  int32_t* status;  // nullable; cleared here (this kernel waits for nothing)
  int T, K, N, out_fp32;
};

constexpr int kStreamWarps = 8;

// Few tokens: a CTA owns 16 weight rows and 8 NT tokens; its warps take the
// 128-column blocks in turn, each streaming weights straight from global
// memory into mma.sync operands (every byte once, 16 per lane), and their sums
// are joined in warp order.  HBM bound: 8 tokens, 7168 x 36864 weights run at
// 5.9 TB/s with four CTAs an SM (64 registers a thread); where the row tiles
// do not even cover the SMs, the latency of a warp's chain counts instead and
// more registers (more loads in flight a warp) win: 8 x 7168 x 2112 4.3 us
// against 5.3.
template <int NT, int MIN_CTAS>
__global__ void __launch_bounds__(32 * kStreamWarps, MIN_CTAS) linear_stream_kernel(const StreamParams p) {
  __shared__ float part[kStreamWarps][NT * 4][32];
  pdl_wait();
  pdl_trigger();
  if (p.status && blockIdx.x == 0 && threadIdx.x < kStatusInts) p.status[threadIdx.x] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16, nb = blocks128(p.K);
  const float* ws = p.ws + (int64_t)(n0 / kBlk) * nb;
  const uint8_t* w0 = p.w + (int64_t)min(n0 + g, p.N - 1) * p.K + 16 * t;  // past N: not stored
  const uint8_t* w1 = p.w + (int64_t)min(n0 + g + 8, p.N - 1) * p.K + 16 * t;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int b = warp; b < nb; b += kStreamWarps) {
    uint4 w[4];
    const int k0 = b * kBlk;
    const bool in[2] = {k0 + 16 * t < p.K, k0 + 16 * t + 64 < p.K};
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = in[j & 1] ? ldg_stream((j < 2 ? w0 : w1) + k0 + 64 * (j & 1)) : zero;
    const float sw = ws[b];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* xr = p.xq + (int64_t)min(8 * i + g, p.T - 1) * p.K + k0 + 16 * t;
      uint4 x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) x[j] = in[j] ? *reinterpret_cast<const uint4*>(xr + 64 * j) : zero;
      const float s0 = sw * p.xs[(int64_t)min(8 * i + 2 * t, p.T - 1) * nb + b];
      const float s1 = sw * p.xs[(int64_t)min(8 * i + 2 * t + 1, p.T - 1) * nb + b];
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_block(d, w, x);
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
    const int tok = o >> 4, r = o & 15, c = tok & 7;
    const int l = 4 * (r & 7) + (c >> 1), j = 4 * (tok >> 3) + 2 * (r >> 3) + (c & 1);
    float v = 0.f;
#pragma unroll
    for (int wq = 0; wq < kStreamWarps; ++wq) v += part[wq][j][l];
    if (tok < p.T && n0 + r < p.N) {
      const int64_t at = (int64_t)tok * p.out_ld + n0 + r;
      if (p.out_fp32)
        static_cast<float*>(p.out)[at] = v;
      else
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rn(v);
    }
  }
}

constexpr int kStreamMaxT = 16;

}  // namespace

size_t linear_fp8_workspace(int, int, int) { return 256; }

// Up to 16 tokens are streamed (measured at 7168 x 7168: 16 tokens 15-17 us
// against 20 us of the tensor-core kernel; at 32 tokens 37 us against 16 us).
cudaError_t launch_linear_fp8(const LinearFp8Args& a, cudaStream_t s) {
  if (a.T > kStreamMaxT) return launch_linear_fp8_tc(a, s);
  const StreamParams p{a.xq, a.w, a.xs, a.ws, a.out, a.out_ld, static_cast<int32_t*>(a.scratch), a.T, a.K, a.N,
                       a.out_fp32 ? 1 : 0};
  const unsigned rows = (unsigned)((a.N + 15) / 16);
  const dim3 grid(rows), block(32 * kStreamWarps);
  if (a.T > 8) return launch_pdl(linear_stream_kernel<2, 1>, grid, block, 0, s, p);
  if (rows <= 152) return launch_pdl(linear_stream_kernel<1, 1>, grid, block, 0, s, p);
  return launch_pdl(linear_stream_kernel<1, 4>, grid, block, 0, s, p);
}

}  // namespace fp4moe
