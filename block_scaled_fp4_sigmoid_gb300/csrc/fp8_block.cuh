// Device helpers of the block-scaled FP8 operators: E4M3 values with one fp32
// scale per row and 128 columns (activations) or per 128 x 128 block
// (weights).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace fp4moe {

constexpr int kBlk = 128;  // columns (and weight rows) of one scale block

__host__ __device__ constexpr int blocks128(int n) { return (n + kBlk - 1) / kBlk; }

// 16 bytes read once (weights): not kept in L1.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Starts `bytes` (a multiple of 16) at p, 16-byte aligned, on their way into L2.  No
// hazard with a kernel that still writes them: L2 is where such writes arrive.
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Two fp32 values from the two bf16 halves of a word.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale of a block: fp32(amax / 448).
__device__ __forceinline__ float e4m3_scale(float amax) { return __fdiv_rn(amax, 448.0f); }

// Codes are RNE_E4M3(fp32(v * r)), saturating, with r = fp32(1 / s) taken once a
// block: a correctly rounded division for each value made the SwiGLU bound by
// its instructions (88 us at 4096 x 18432).  Scales below the
// normal range, whose reciprocal may not be finite, divide.  A scale that is
// not positive (an all-zero block, or a NaN in it) gives signed zeros, and NaN
// where v is NaN.
__device__ __forceinline__ float e4m3_scaled(float v, float s, float r) {
  if (s >= 1.17549435e-38f) return v * r;
  return s > 0.f ? __fdiv_rn(v, s) : v * 0.f;
}

// E4M3 codes of four scaled values, value j in byte j.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// silu(g) * u with the hardware base-2 exponential (results below the normal
// range flush to zero: 1 + e^-g is 1 then) and reciprocal.
__device__ __forceinline__ float swiglu(float g, float u) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  return g * rcp_approx(1.f + e) * u;
}

// d += A (16 x 32) . B (32 x 8), E4M3 inputs, fp32 accumulation.  With lane =
// 4 g + t: a0, a2 from row g, a1, a3 from row g + 8, b0, b1 from column g;
// d0, d1 are row g and columns 2t, 2t + 1, d2, d3 the same of row g + 8.  The
// sum over K does not depend on which K index a lane's bytes carry as long
// as A and B agree, so a lane takes 16 consecutive bytes of its row and its
// column and feeds words 0, 1 to one instruction and 2, 3 to the next.
__device__ __forceinline__ void mma_e4m3(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One 128-column block: 16 weight rows against 8 columns; w[0..1] are row g's
// two 16-byte pieces (64 columns apart), w[2..3] row g + 8's, x[0..1] column g's.
__device__ __forceinline__ void mma_block(float* d, const uint4* w, const uint4* x) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    mma_e4m3(d, w[j].x, w[2 + j].x, w[j].y, w[2 + j].y, x[j].x, x[j].y);
    mma_e4m3(d, w[j].z, w[2 + j].z, w[j].w, w[2 + j].w, x[j].z, x[j].w);
  }
}

}  // namespace fp4moe
