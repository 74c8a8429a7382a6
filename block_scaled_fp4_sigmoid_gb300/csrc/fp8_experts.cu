// Block-scaled FP8 experts for few tokens, in two kernels: gate/up + SwiGLU +
// E4M3 requantisation, then down + weighted combine.
//
// The columns of the MMAs are tokens: an entry of the list is a chosen expert
// with up to 8 of the tokens that chose it (T <= 8: column = token; more
// tokens: the set ones in order, two entries where more than 8 chose it), so
// an expert's weights are read once for 8 tokens, and both kernels only visit
// experts that some token chose.
#include <algorithm>

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4moe {

namespace {

constexpr int kMaxE = kExpertsMaxE, kMaxTok = kExpertsMaxT, kMaxRoutes = kExpertsMaxK * kMaxTok;
constexpr int kMaxList = kMaxRoutes + 2;  // entries: at most one a route, and the shared expert's two
constexpr int kNoTok = 255;

struct ExpertsParams {
  const uint8_t *xq, *w13, *w2, *sh13, *sh2;
  const float *xs, *s13, *s2, *ss13, *ss2;
  const int32_t* idx;
  const float* wts;
  uint8_t* hq;   // [entry * 8 + column, I]
  float* hs;     // [entry * 8 + column, I / 128]
  uint16_t* out;
  int T, H, I, E, k, shared;
  int split;   // CTAs that share a gate/up unit
  int dsplit;  // CTAs that share 16 output columns
};

struct ExpertList {
  uint32_t mask[kMaxE + 1];    // tokens that chose the expert
  uint16_t e[kMaxList];        // entries by ascending expert; the shared one is E
  uint8_t tok[kMaxList][8];    // token of each column, or kNoTok
  uint8_t cols[kMaxList];      // bit c: column c has a token
  int16_t route[kMaxRoutes];   // expert of each (token, slot), -1: none here
  int n;
};

// Lists the chosen experts; both kernels of a call get the same list.  Routes
// outside [0, E) (an expert that another rank holds) choose nothing.
__device__ __forceinline__ void list_experts(const ExpertsParams& p, ExpertList& L) {
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) L.mask[e] = 0u;
  __syncthreads();
  for (int r = threadIdx.x; r < p.T * p.k; r += blockDim.x) {
    const int e = p.idx[r];
    const bool in = e >= 0 && e < p.E;
    L.route[r] = (int16_t)(in ? e : -1);
    if (in) atomicOr(&L.mask[e], 1u << (r / p.k));
  }
  if (threadIdx.x == 0 && p.shared) L.mask[p.E] = (1u << p.T) - 1u;
  __syncthreads();
  if (threadIdx.x < 32) {
    int n = 0;
    const uint32_t below = (1u << threadIdx.x) - 1u;
    for (int e0 = 0; e0 <= p.E; e0 += 32) {
      const int e = e0 + threadIdx.x;
      const int cnt = e <= p.E ? __popc(L.mask[e]) : 0;
      const uint32_t one = __ballot_sync(0xffffffffu, cnt > 0), two = __ballot_sync(0xffffffffu, cnt > 8);
      const int at = n + __popc(one & below) + __popc(two & below);
      if (cnt > 0) L.e[at] = (uint16_t)e;
      if (cnt > 8) L.e[at + 1] = (uint16_t)e;
      n += __popc(one) + __popc(two);
    }
    if (threadIdx.x == 0) L.n = n;
  }
  __syncthreads();
  for (int o = threadIdx.x; o < L.n * 8; o += blockDim.x) {
    const int u = o >> 3, c = o & 7, e = L.e[u];
    uint32_t m = L.mask[e];
    int tok = kNoTok;
    if (p.T <= 8) {
      if ((m >> c) & 1u) tok = c;
    } else {  // the set bit of this place; an expert's second entry goes on after eight
      const int nth = c + (u > 0 && L.e[u - 1] == e ? 8 : 0);
      if (nth < __popc(m)) {
        for (int i = 0; i < nth; ++i) m &= m - 1u;
        tok = __ffs(m) - 1;
      }
    }
    L.tok[u][c] = (uint8_t)tok;
    if (c == 0) {
      const int n = __popc(L.mask[e]), before = p.T > 8 && u > 0 && L.e[u - 1] == e ? 8 : 0;
      L.cols[u] = (uint8_t)(p.T <= 8 ? L.mask[e] : (1u << min(8, n - before)) - 1u);
    }
  }
  __syncthreads();
}

constexpr int kGuThreads = 512;

// The two halves of cluster_arrive_wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A word to this CTA's shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, int rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\tst.shared::cluster.f32 [ra], %2;\n\t}" ::"r"(addr),
      "r"(rank), "f"(v)
      : "memory");
}

// One unit: 128 gate and 128 up rows (one scale block of h) of one entry.
// Warp = 16 gate rows and the 16 up rows of the same h values, over every
// second K block, straight from global memory into mma.sync operands: 8 loads
// of 16 bytes in flight a lane.  HBM bound: 8 tokens over 384 experts (1.75
// GB) in 262 us, 6.7 TB/s.
//
// SPLIT: a unit is shared by a cluster, each CTA with every split-th pair of K
// blocks; CTA 0 gets the others' sums in its shared memory and finishes.
template <bool SPLIT>
__global__ void __launch_bounds__(kGuThreads, 1) experts_gateup_kernel(const ExpertsParams p) {
  extern __shared__ __align__(16) float others[];  // SPLIT: [split - 1][8 warps][8][32]
  __shared__ ExpertList L;
  __shared__ float part[8][8][32];
  __shared__ float amax[8][8];
  __shared__ __align__(16) uint8_t codes[8][128];  // read as 16-byte words
  pdl_wait();
  pdl_trigger();
  list_experts(p, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rg = warp & 7, kh = warp >> 3;
  const int S = SPLIT ? p.split : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
  const int hb = p.H / kBlk, ib = p.I / kBlk, units = L.n * ib;
  if constexpr (SPLIT) cluster_arrive();
  for (int unit = (int)blockIdx.x / S; unit < units; unit += (int)gridDim.x / S) {
    const int u = unit / ib, b = unit - u * ib, e = L.e[u];
    const bool sh = e == p.E;
    const uint8_t* w = sh ? p.sh13 : p.w13 + (int64_t)e * 2 * p.I * p.H;
    const float* ws = sh ? p.ss13 : p.s13 + (int64_t)e * 2 * ib * hb;
    const uint8_t* row = w + (int64_t)(b * kBlk + 16 * rg + g) * p.H;
    const float *wsg = ws + (int64_t)b * hb, *wsu = ws + (int64_t)(ib + b) * hb;
    // columns without a token compute token 0's values, which go nowhere
    auto tok_of = [&](int c) { return L.tok[u][c] == kNoTok ? 0 : (int)L.tok[u][c]; };
    const uint8_t* xr = p.xq + (int64_t)tok_of(g) * p.H;
    const float *xs0 = p.xs + (int64_t)tok_of(2 * t) * hb, *xs1 = p.xs + (int64_t)tok_of(2 * t + 1) * hb;
    float acc[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
#pragma unroll 1
    for (int kb = 2 * rank + kh; kb < hb; kb += 2 * S) {
      uint4 wv[2][4], x[2];
      const int64_t k0 = kb * kBlk + 16 * t;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          wv[m][j] = ldg_stream(row + (int64_t)(m * p.I + 8 * (j >> 1)) * p.H + k0 + 64 * (j & 1));
      const float sw[2] = {wsg[kb], wsu[kb]};
      x[0] = *reinterpret_cast<const uint4*>(xr + k0);
      x[1] = *reinterpret_cast<const uint4*>(xr + k0 + 64);
      const float x0 = xs0[kb], x1 = xs1[kb];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_block(d, wv[m], x);
        const float s0 = sw[m] * x0, s1 = sw[m] * x1;
        acc[m][0] = fmaf(s0, d[0], acc[m][0]);
        acc[m][1] = fmaf(s1, d[1], acc[m][1]);
        acc[m][2] = fmaf(s0, d[2], acc[m][2]);
        acc[m][3] = fmaf(s1, d[3], acc[m][3]);
      }
    }
    // the odd K blocks' sums join the even ones'
    if (kh) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[rg][m * 4 + j][lane] = acc[m][j];
    }
    __syncthreads();
    if constexpr (SPLIT) {
      if (!kh) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][j] += part[rg][m * 4 + j][lane];
      }
      cluster_wait();  // every CTA has begun, and CTA 0 has read the unit before
      if (!kh && rank > 0) {
        const uint32_t at = smem_u32(others + (((rank - 1) * 8 + rg) * 8) * 32 + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) st_cluster(at + 128u * i, 0, acc[i >> 2][i & 3]);
      }
      __syncwarp();
      cluster_arrive_wait();
      if (!kh && rank == 0) {
        for (int r = 0; r < S - 1; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] += others[((r * 8 + rg) * 8 + i) * 32 + lane];
      }
      __syncwarp();
      cluster_arrive();
      if (rank > 0) continue;
    }
    float h[4];
    if (!kh) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = SPLIT ? swiglu(acc[0][j], acc[1][j])
                     : swiglu(acc[0][j] + part[rg][j][lane], acc[1][j] + part[rg][4 + j][lane]);
      // columns 2t (j = 0, 2) and 2t + 1: largest |h| over the warp's 16 rows
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float a = max_nan(fabsf(h[c]), fabsf(h[c + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (g == 0) amax[rg][2 * t + c] = a;
      }
    }
    __syncthreads();
    if (!kh) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 2 * t + c;
        float a = amax[0][col];
#pragma unroll
        for (int q = 1; q < 8; ++q) a = max_nan(a, amax[q][col]);
        const float s = e4m3_scale(a), r = __fdiv_rn(1.f, s);
        const uint32_t two = e4m3x4(e4m3_scaled(h[c], s, r), e4m3_scaled(h[c + 2], s, r), 0.f, 0.f);
        codes[col][16 * rg + g] = (uint8_t)two;
        codes[col][16 * rg + g + 8] = (uint8_t)(two >> 8);
        if (rg == 0 && g == 0) p.hs[(int64_t)(u * 8 + col) * ib + b] = s;
      }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 64; o += kGuThreads) {
      const int col = o >> 3, c = 16 * (o & 7);
      if (L.tok[u][col] != kNoTok)
        *reinterpret_cast<uint4*>(p.hq + (int64_t)(u * 8 + col) * p.I + b * kBlk + c) =
            *reinterpret_cast<const uint4*>(&codes[col][c]);
    }
  }
  if constexpr (SPLIT) cluster_wait();
}

// How many clusters of `split` CTAs run at the same time.
int64_t clusters_of(int split) { return split == 1 ? 152 : split == 2 ? 76 : split == 4 ? 36 : 15; }

// How many CTAs share a gate/up unit, by the rounds of units and a unit's time:
// an SM takes a K block in 0.42 us, a join 1.5 us.  Measured (calls; 1, 2, 4, 8 CTAs):
// 4 units of 56 K blocks 33, 23, 16, 13 us; 30 of 56: 39, 28, 23, 26; 64 of 56: 43,
// 34, 37, 46; 88 of 22: 29, 35, 35, 45; 128 of 8: 14, 18, 20, 31.
int gateup_split(int64_t units, int hb) {
  int best = 1;
  int64_t cost = (units + clusters_of(1) - 1) / clusters_of(1) * hb * 42;  // 10 ns
  for (int s = 2; s <= 8; s *= 2) {
    const int64_t c = (units + clusters_of(s) - 1) / clusters_of(s) * ((hb + 2 * s - 1) / (2 * s) * 84 + 150);
    if (c < cost) cost = c, best = s;
  }
  return best;
}

// One CTA: 16 output columns (rows of every chosen expert's W2), all tokens.
// Runs of two K blocks go to the warps in turn, over all entries; a warp adds
// weight * scales * product to its token columns, and the warps' sums are
// joined in warp order, so the result does not depend on timing (SPLIT: a cluster's
// CTAs share the runs, and CTA 0 joins their sums in its order).  A warp's sums
// are in registers where column = token (T <= 8), else in its own shared memory
// (GATHER).
//
// HBM bound, 6.3 to 6.6 TB/s over both kernels at 8 tokens and 384 experts (398 to
// 417 us on several machines for 2.6 GB).  All loads of a run are issued together, 24 warps an SM: with one K
// block a run the call took 428 us, with four (16 warps) 421, with one prefetched
// a block ahead 435, with blocks copied ahead into shared memory by cp.async 485
// and more.
//
// The gate/up kernel has passed its own wait before this one can start, so all
// but its output (h) is complete: the list and the routing weights are made
// before the wait.
template <bool GATHER, int kDnWarps, bool SPLIT>
__global__ void __launch_bounds__(32 * kDnWarps, 24 / kDnWarps) experts_down_kernel(const ExpertsParams p) {
  __shared__ ExpertList L;
  __shared__ float rw[kMaxList][8];  // routing weight of (entry, column)
  __shared__ float sums[kDnWarps][16][GATHER ? 17 : 9];  // row, token
  __shared__ float others[SPLIT ? 3 : 1][16 * kMaxTok];  // SPLIT: the other CTAs' sums
  const int S = SPLIT ? p.dsplit : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
  if constexpr (SPLIT) cluster_arrive();
  list_experts(p, L);
  for (int o = threadIdx.x; o < L.n * 8; o += blockDim.x) {
    const int u = o >> 3, tok = L.tok[u][o & 7], e = L.e[u];
    float v = 0.f;
    if (tok != kNoTok) {
      if (e == p.E) v = 1.f;
      else
        for (int j = 0; j < p.k; ++j)  // (an expert chosen twice: its weights add)
          if (L.route[tok * p.k + j] == e) v += p.wts[tok * p.k + j];
    }
    rw[u][o & 7] = v;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if constexpr (GATHER)
    for (int o = lane; o < 16 * 17; o += 32) sums[warp][0][o] = 0.f;
  __syncthreads();
  const int n0 = (int)blockIdx.x / S * 16, hb = p.H / kBlk, ib = p.I / kBlk;
  const int64_t wat = (int64_t)(n0 + g) * p.I + 16 * t, sat = (int64_t)(n0 / kBlk) * ib;  // into an expert's weights, scales
  constexpr int kRun = 2;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  // a warp takes every S kDnWarps-th run of kRun K blocks, over all entries
  const int runs = (ib + kRun - 1) / kRun;
  int u = 0, r = rank * kDnWarps + warp;
  pdl_wait();
  pdl_trigger();
  for (;; r += S * kDnWarps) {
    while (r >= runs) r -= runs, ++u;
    if (u >= L.n) break;
    const int e = L.e[u], b0 = r * kRun;
    const uint32_t cols = L.cols[u];
    const bool sh = e == p.E;
    const uint8_t* w = (sh ? p.sh2 : p.w2 + (int64_t)e * p.H * p.I) + wat + b0 * kBlk;
    const float* ws = (sh ? p.ss2 : p.s2 + (int64_t)e * hb * ib) + sat + b0;
    const uint8_t* h = p.hq + (int64_t)(u * 8 + g) * p.I + b0 * kBlk + 16 * t;
    const float* hs = p.hs + (int64_t)(u * 8 + 2 * t) * ib + b0;
    uint4 wv[kRun][4], hv[kRun][2];
    float s[kRun][2];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const bool in = b0 + k < ib;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        wv[k][j] = in ? ldg_stream(w + (int64_t)8 * (j >> 1) * p.I + 64 * (j & 1) + k * kBlk) : make_uint4(0, 0, 0, 0);
      // a column without a token has no h: it is zero and adds nothing (not
      // even a NaN of the weights)
      hv[k][0] = hv[k][1] = make_uint4(0, 0, 0, 0);
      if (in && ((cols >> g) & 1u)) {
        hv[k][0] = *reinterpret_cast<const uint4*>(h + k * kBlk);
        hv[k][1] = *reinterpret_cast<const uint4*>(h + k * kBlk + 64);
      }
      const float sw = in ? ws[k] : 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) s[k][c] = in && ((cols >> (2 * t + c)) & 1u) ? sw * hs[c * ib + k] : 0.f;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_block(d, wv[k], hv[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = fmaf(s[k][j & 1], d[j], sum[j]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if ((cols >> (2 * t + c)) & 1u) {
        const float f = rw[u][2 * t + c];
        if constexpr (GATHER) {  // a column's (row, token) is this lane's alone
          const int tok = L.tok[u][2 * t + c];
          sums[warp][g][tok] = fmaf(f, sum[c], sums[warp][g][tok]);
          sums[warp][g + 8][tok] = fmaf(f, sum[c + 2], sums[warp][g + 8][tok]);
        } else {
          acc[c] = fmaf(f, sum[c], acc[c]);
          acc[c + 2] = fmaf(f, sum[c + 2], acc[c + 2]);
        }
      }
    if constexpr (GATHER) __syncwarp();  // the next run may bring the token in another column
  }
  if constexpr (!GATHER) {
    sums[warp][g][2 * t] = acc[0], sums[warp][g][2 * t + 1] = acc[1];
    sums[warp][g + 8][2 * t] = acc[2], sums[warp][g + 8][2 * t + 1] = acc[3];
  }
  __syncthreads();
  if constexpr (SPLIT) {
    static_assert(32 * kDnWarps >= 16 * kMaxTok, "an output a thread");
    const int o = threadIdx.x, tok = o >> 4, row = o & 15;
    float v = 0.f;
    if (o < 16 * p.T) {
#pragma unroll
      for (int wq = 0; wq < kDnWarps; ++wq) v += sums[wq][row][tok];
    }
    __syncwarp();
    cluster_wait();  // every CTA has begun
    if (rank > 0 && o < 16 * p.T) st_cluster(smem_u32(&others[rank - 1][o]), 0, v);
    __syncwarp();
    cluster_arrive_wait();
    if (rank == 0 && o < 16 * p.T) {
      for (int q = 0; q < S - 1; ++q) v += others[q][o];
      p.out[(int64_t)tok * p.H + n0 + row] = f32_to_bf16_rn(v);
    }
    return;
  }
  for (int o = threadIdx.x; o < 16 * p.T; o += 32 * kDnWarps) {
    const int tok = o >> 4, r = o & 15;
    float v = 0.f;
#pragma unroll
    for (int wq = 0; wq < kDnWarps; ++wq) v += sums[wq][r][tok];
    p.out[(int64_t)tok * p.H + n0 + r] = f32_to_bf16_rn(v);
  }
}

// How many CTAs share 16 output columns of the down kernel, by the K blocks over all
// entries and the number of such column groups.  24 warps take 48 K blocks in about
// 1 us, a join 1.5 us (two CTAs) or 2.2 (four).  Measured (calls; 1, 2, 4 CTAs): 16
// tokens, 76 entries, H 256, I 2048 53, 39, 33 us; H 512, I 512 22, 19, 20; H 1024, I
// 2048 76, 64 us; 4 tokens, 16 entries, H 512, I 2048 21, 19, 18; I 512 9, 10, 12.
int down_split(int64_t blocks, int64_t cols) {
  int best = 1;
  int64_t cost = blocks * 100 / 48;  // 10 ns
  for (int s = 2; s <= 4; s *= 2) {
    const int64_t c = blocks * 100 / (48 * s) + (s == 2 ? 150 : 220);
    if (cols <= clusters_of(s) && c < cost) cost = c, best = s;
  }
  return best;
}

// Entries of the list: an expert with c tokens has ceil(c / 8) <= 1 + c / 8.
int64_t list_cap(const fp4moe_dims& d) {
  const int routes = d.T * d.top_k;
  return std::min(d.E, routes) + (d.T > 8 ? routes / 8 : 0) + d.n_shared * ((d.T + 7) / 8);
}

int64_t hq_bytes(const fp4moe_dims& d) { return list_cap(d) * 8 * d.I; }  // a multiple of 1024

}  // namespace

size_t experts_fp8_workspace(const fp4moe_dims& d) {
  return (size_t)std::max<int64_t>(256, hq_bytes(d) + list_cap(d) * 8 * (d.I / kBlk) * 4);  // (0 says: unsupported)
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
  // one CTA fills an SM's registers; its units follow each other
  const int64_t units = list_cap(d) * (d.I / kBlk);
  p.split = gateup_split(units, d.H / kBlk);
  cudaError_t e;
  if (p.split > 1) {
    const int64_t n = std::min(units, clusters_of(p.split));
    const size_t smem = (size_t)(p.split - 1) * 8 * 8 * 32 * sizeof(float);
    e = cudaFuncSetAttribute(experts_gateup_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 7 * 8192);
    if (e == cudaSuccess)
      e = launch_pdl_cluster(experts_gateup_kernel<true>, dim3((unsigned)(n * p.split)), dim3(kGuThreads), smem, s,
                             (unsigned)p.split, p);
  } else {
    e = launch_pdl(experts_gateup_kernel<false>, dim3((unsigned)std::min<int64_t>(units, sms)), dim3(kGuThreads), 0, s, p);
  }
  if (e != cudaSuccess) return e;
  p.dsplit = down_split(list_cap(d) * (d.I / kBlk), d.H / 16);
  const unsigned cols = (unsigned)(d.H / 16);
  if (p.dsplit > 1)
    return launch_pdl_cluster(d.T <= 8 ? experts_down_kernel<false, 24, true> : experts_down_kernel<true, 24, true>,
                              dim3(cols * p.dsplit), dim3(768), 0, s, (unsigned)p.dsplit, p);
  // an SM runs 24 warps of the down kernel: as one CTA where the output columns
  // make at most two a SM (8 tokens, H = 1024, I = 512, 32 experts: 14 us a call
  // against 20), else as three (one token, H = 7168: 68 us against 75)
  if (cols <= 2u * sms)
    return launch_pdl(d.T <= 8 ? experts_down_kernel<false, 24, false> : experts_down_kernel<true, 24, false>, dim3(cols),
                      dim3(768), 0, s, p);
  return launch_pdl(d.T <= 8 ? experts_down_kernel<false, 8, false> : experts_down_kernel<true, 8, false>, dim3(cols),
                    dim3(256), 0, s, p);
}

}  // namespace fp4moe
