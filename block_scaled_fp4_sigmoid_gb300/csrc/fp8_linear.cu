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
  int32_t* status;  // nullable; cleared here (this kernel waits for nothing)
  int T, K, N, out_fp32;
  int ahead;  // fetch weights ahead of the wait
};

constexpr int kStreamWarps = 8;

// A CTA owns 16 weight rows and 8 NT tokens; its warps take runs of
// RUN 128-column blocks in turn, all loads of a run issued together, straight
// from global memory into mma.sync operands (every weight byte once, 16 per
// lane), and their sums are joined in warp order.  HBM bound: 8 tokens and 7168
// x 36864 weights in 42 us, 6.3 TB/s.
//
// Weights fetched into L2 before the wait for the launch before: 44.1 -> 42.0 us, 4
// x 4096 x 4096 4.8 -> 3.9, 16 x 7168 x 2112 6.8 -> 6.3; for up to 8 tokens and a CTA an
// SM at most it does not pay (1 x 7168 x 2112 4.0 -> 4.3).  Fetched ahead inside the
// loop too: 53 to 63 us.
template <int NT, int MIN_CTAS, int RUN>
__global__ void __launch_bounds__(32 * kStreamWarps, MIN_CTAS) linear_stream_kernel(const StreamParams p) {
  __shared__ float part[kStreamWarps][NT * 4][32];
  {
    // the first run's weights on their way into L2 while the launch before ends
    const int row = min((int)blockIdx.x * 16 + ((int)threadIdx.x & 15), p.N - 1), b = ((int)threadIdx.x >> 5) * RUN;
    const int n = min(RUN * kBlk, p.K - b * kBlk);
    if (p.ahead && (threadIdx.x & 31) < 16 && n > 0) prefetch_l2(p.w + (int64_t)row * p.K + b * kBlk, n);
  }
  pdl_wait();
  pdl_trigger();
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kStatusInts) p.status[threadIdx.x] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * (8 * NT), nb = blocks128(p.K);
  const float* ws = p.ws + (int64_t)(n0 / kBlk) * nb;
  const uint8_t* w0 = p.w + (int64_t)min(n0 + g, p.N - 1) * p.K + 16 * t;  // past N: not stored
  const uint8_t* w1 = p.w + (int64_t)min(n0 + g + 8, p.N - 1) * p.K + 16 * t;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 1
  for (int b0 = warp * RUN; b0 < nb; b0 += kStreamWarps * RUN) {
    uint4 w[RUN][4];
    float sw[RUN];
    bool in[RUN][2];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      const int k0 = (b0 + r) * kBlk;
#pragma unroll
      for (int j = 0; j < 2; ++j) in[r][j] = k0 + 16 * t + 64 * j < p.K;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[r][j] = in[r][j & 1] ? ldg_stream((j < 2 ? w0 : w1) + k0 + 64 * (j & 1)) : zero;
      sw[r] = ws[min(b0 + r, nb - 1)];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* xr = p.xq + (int64_t)min(t0 + 8 * i + g, p.T - 1) * p.K + b0 * kBlk + 16 * t;
      const float* xs0 = p.xs + (int64_t)min(t0 + 8 * i + 2 * t, p.T - 1) * nb;
      const float* xs1 = p.xs + (int64_t)min(t0 + 8 * i + 2 * t + 1, p.T - 1) * nb;
#pragma unroll
      for (int r = 0; r < RUN; ++r) {
        uint4 x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) x[j] = in[r][j] ? *reinterpret_cast<const uint4*>(xr + r * kBlk + 64 * j) : zero;
        const int b = min(b0 + r, nb - 1);
        // (a block past the end: its product is exactly zero, whatever the scales are not NaN)
        const float s0 = b0 + r < nb ? sw[r] * xs0[b] : 0.f, s1 = b0 + r < nb ? sw[r] * xs1[b] : 0.f;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_block(d, w[r], x);
        acc[i][0] = fmaf(s0, d[0], acc[i][0]);
        acc[i][1] = fmaf(s1, d[1], acc[i][1]);
        acc[i][2] = fmaf(s0, d[2], acc[i][2]);
        acc[i][3] = fmaf(s1, d[3], acc[i][3]);
      }
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

// Weights streamed into mma.sync, or through shared memory into the tensor cores:
// the former starts 1 to 2 us sooner, the latter has no rounds of CTAs each with a
// latency of its own, and reads the weights once where the former reads them for
// every 16 tokens.  Up to 128 tokens the smaller of two estimates decides, both
// fitted to measurements (stream, tensor cores): 8 x 7168 x 36864 42.0, 42.4 us;
// 8 x 1024 x 131072 36.7, 26.8; 16 x 7168 x 36864 74.7, 42.1; 16 x 7168 x 2112 6.3,
// 7.8; 64 x 2048 x 512 2.7, 4.9; 32 x 7168 x 2112 12.5, 7.9.  This is the estimate of
// the stream, in units of 10 ns.
static int64_t stream_cost(int T, int K, int N) {
  const int64_t sms = 152, nb = blocks128(K), ctas = (N + 15) / 16 * (T > 8 ? (T + 15) / 16 : 1);
  const int64_t rounds = (ctas + 3 * sms - 1) / (3 * sms);  // of three CTAs an SM
  if (T > 8) return ctas <= sms ? 160 + nb * 7 : rounds * (150 + nb * 19);
  return std::max(ctas <= 2 * sms ? 150 + nb * 5 : (ctas <= 4 * sms ? 1 : rounds) * (140 + nb * 8), (int64_t)K * N / 60000);  // (6 TB/s)
}

// The instance of linear_stream_kernel for a call, or the tensor cores.
struct StreamChoice {
  int nt, min_ctas, run;  // nt = 0: the tensor cores
  bool ahead;
  const char* name;
};

// The more CTAs share an SM, the fewer registers and so the fewer loads in
// flight a warp.  With row tiles for all of them, two blocks a run and three CTAs
// an SM stream best, unless the last round of CTAs would be much emptier than
// with one block and four CTAs (7168 x 7168, 448 tiles, 8 tokens: 11.0 us against
// 11.9; 7168 x 36864, 2304 tiles: 49.6 against 44.1).  Where the tiles hardly
// cover the SMs, four blocks a run (7168 x 2112, 132 tiles: 4.4 us against 5.2;
// 16 tokens 6.9 against 10.1).
static StreamChoice stream_choice(int T, int K, int N) {
  const int64_t rows = (N + 15) / 16, sms = 152;
  const int64_t ctas = rows * (T > 8 ? (T + 15) / 16 : 1);
  if (T > 128) return {0, 0, 0, false, ""};
  const int64_t stream = stream_cost(T, K, N) - 250;  // (what the tensor cores start later)
  if (stream > (int64_t)K * N / 56000 && stream > linear_fp8_tc_cost(T, K, N)) return {0, 0, 0, false, ""};
  if (T > 8) {
    if (ctas <= sms) return {2, 1, 4, true, "stream 2x1x4 ahead"};
    return {2, 3, 2, true, "stream 2x3x2 ahead"};
  }
  if (ctas <= sms) return {1, 2, 4, false, "stream 1x2x4"};
  if (ctas <= 2 * sms) return {1, 2, 4, true, "stream 1x2x4 ahead"};
  const int64_t at3 = (ctas + 3 * sms - 1) / (3 * sms) * 3, at4 = (ctas + 4 * sms - 1) / (4 * sms) * 4;  // CTA slots
  if (at3 <= at4) return {1, 3, 2, true, "stream 1x3x2 ahead"};
  return {1, 4, 1, true, "stream 1x4x1 ahead"};
}

const char* linear_fp8_form(int T, int K, int N) {
  const StreamChoice c = stream_choice(T, K, N);
  return c.nt ? c.name : linear_fp8_tc_form(T, K, N);
}

cudaError_t launch_linear_fp8(const LinearFp8Args& a, cudaStream_t s) {
  const StreamChoice c = stream_choice(a.T, a.K, a.N);
  if (c.nt == 0) return launch_linear_fp8_tc(a, s);
  const StreamParams p{a.xq, a.w, a.xs, a.ws, a.out, a.out_ld, static_cast<int32_t*>(a.scratch), a.T, a.K, a.N,
                       a.out_fp32 ? 1 : 0, c.ahead};
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.T + 8 * c.nt - 1) / (8 * c.nt))), block(32 * kStreamWarps);
  switch (100 * c.nt + 10 * c.min_ctas + c.run) {
    case 214: return launch_pdl(linear_stream_kernel<2, 1, 4>, grid, block, 0, s, p);
    case 232: return launch_pdl(linear_stream_kernel<2, 3, 2>, grid, block, 0, s, p);
    case 124: return launch_pdl(linear_stream_kernel<1, 2, 4>, grid, block, 0, s, p);
    case 132: return launch_pdl(linear_stream_kernel<1, 3, 2>, grid, block, 0, s, p);
    default: return launch_pdl(linear_stream_kernel<1, 4, 1>, grid, block, 0, s, p);
  }
}

}  // namespace fp4moe
