// The paged key-value cache on the device: addresses, a row's sequence and
// position, what a position sees, and the finished rows of attention.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fp8_block.cuh"

namespace fp4moe {

constexpr int kPageStep = 16;  // tokens that share a page wherever they start (the smallest page)

struct PagedKv {
  uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;  // bytes
  int pages, page_shift, heads;
};

struct PagedBatch {
  const int32_t *starts, *lens, *table;
  int64_t table_ld;
  int rows, seqs, reach;  // reach: tokens that a row of the table lists
};

// What finished rows go to: bf16, or E4M3 codes with a scale per 128 columns.
struct PagedOut {
  uint16_t* out;
  uint8_t* codes;
  float* scales;
  int cols;  // q_heads * head_dim
};

struct PagedAttn {
  PagedKv kv;
  PagedBatch batch;
  PagedOut out;
  const uint16_t* q;
  int64_t q_ld;
  int q_heads, group;  // group: query heads a key-value head
  int window, sinks;
  float scale_log2;  // scale * log2(e): softmax in base 2
};

// Page of sequence b's tokens from position p < reach on; negative for a hole.
__device__ __forceinline__ int page_of(const PagedKv& kv, const PagedBatch& bt, int b, int p) {
  const int page = bt.table[b * bt.table_ld + (p >> kv.page_shift)];
  return (unsigned)page < (unsigned)kv.pages ? page : -1;
}

// The sequence of `row`: the last b with starts[b] <= row (warp-wide, 32 probes
// a step); -1 where no sequence has it.
__device__ __forceinline__ int seq_of_row(const PagedBatch& bt, int row, int lane) {
  if (!bt.starts) return row < bt.seqs ? row : -1;
  int lo = 0, hi = bt.seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, i < hi && bt.starts[i] <= row);
    const int c = m ? 31 - __clz(m) : 0;
    lo += c * step;
    hi = min(hi, lo + step);
  }
  return bt.starts[lo] <= row && row < bt.starts[lo + 1] ? lo : -1;
}

// Keys that position p sees: [0, sinks) and [lo, n); none (n = 0) from a position
// below 0 or past the table's reach.  Else lo < n.
struct Seen {
  int lo, sinks, n;
};
__device__ __forceinline__ Seen seen_from(int64_t p, int reach, int window, int sinks) {
  Seen s;
  s.n = p >= 0 && p < reach ? (int)p + 1 : 0;
  s.lo = window > 0 ? max(0, s.n - window) : 0;
  s.sinks = min(sinks, s.n);
  return s;
}
__device__ __forceinline__ bool sees(const Seen& s, int j) { return j < s.n && (j >= s.lo || j < s.sinks); }

// 2^x; 0 for -inf.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Softmax weights as fp16 operands for V out of an E4M3 cache.  fp16 has 11 bits where bf16 has 8, but its smallest
// step is 2^-24: many small weights matter together, so they come here scaled by a power of two that brings the largest to 2^15
// (the sums are in the same scale, which the division takes out).  At scores past 2^24 the scale's exponent is rounded:
// the largest weight saturates then.
__device__ __forceinline__ uint32_t f16x2_weights(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four fp32 values of four E4M3 codes.
__device__ __forceinline__ float4 e4m3x4_values(uint32_t w) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  float4 v;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(lo));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(v.z), "=f"(v.w)
      : "r"(hi));
  return v;
}

// A warp's 128 finished columns of one row from column `col` (a multiple of
// 128) on, four a lane; `width` of them exist (64 where one head of 64 is left).
__device__ __forceinline__ void store_cols128(const PagedOut& o, int64_t row, int col, int width, int lane, float4 v) {
  const bool in = 4 * lane < width;
  if (o.out) {
    if (in)
      *reinterpret_cast<uint2*>(o.out + row * o.cols + col + 4 * lane) = make_uint2(bf16x2_rn(v.x, v.y), bf16x2_rn(v.z, v.w));
    return;
  }
  float amax = max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
#pragma unroll
  for (int s = 16; s; s >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, s));
  const float s = e4m3_scale(amax), r = __fdiv_rn(1.f, s);
  if (in)
    *reinterpret_cast<uint32_t*>(o.codes + row * o.cols + col + 4 * lane) =
        e4m3x4(e4m3_scaled(v.x, s, r), e4m3_scaled(v.y, s, r), e4m3_scaled(v.z, s, r), e4m3_scaled(v.w, s, r));
  if (lane == 0) o.scales[row * (o.cols >> 7) + (col >> 7)] = s;
}

}  // namespace fp4moe
