// Causal attention of prompts and prompt chunks over the paged cache, on the
// tensor cores (tcgen05).
//
// A CTA takes two tiles of 128 rows of one key-value head: consecutive tokens of one
// sequence, each with all the query heads that share the head, so that every
// key and value is read once for them all.  For each 128 cached tokens in sight:
//   S = Q K^T into tensor memory (K by TMA, a box a page),
//   P = 2^(S scale - m) in registers, a row a thread: the running maximum m and the sum
//       need no exchange; P goes back over S as 16-bit operands,
//   O += P V in tensor memory, P as the A operand.
// The two tiles take turns: while one's softmax runs on its four warps, the tensor core
// works for the other.  O is rescaled only when a row's maximum has grown by
// 2^8 or more: until then P just grows beyond 1, which costs no precision in
// floating point; the sum is in the same scale and all is divided at the end.
//
// What bounds it: heads of 128, a tile's own chain: 1400 cycles of softmax and 1024 of MMAs and the
// waits between, where the two tiles' MMAs alone would take 2048 (8192 rows of 32 heads: 311 us,
// 1770 TFLOP/s, replayed from a graph a dozen times; 340 to 350 us in long runs of calls, where the power
// cap lowers the clock; the other times here are of graphs too).  So P goes to P V in three parts, the first while the rest is
// computed (whole halves: 326 us).  Tensor memory is full then: 2 S and 2 O of 128 columns.  Heads of 64
// have room for a third S (24 heads, window of 1024, 3 sequences of up to 6001: 130 us, with two 142).  There no
// pipe is full (tensor cores and exponentials a third, issue half): eight warps' chains of wait, fetch, maximum,
// exponentials and store bound it, and the starts and ends of pieces of some ten tiles.  16 softmax warps, half a
// row a thread, were slower (371 us): the halves of a row have to tell each other their maximum.
//
// P is rounded to bf16, an operand's type, for P V (the row's sum has it unrounded): 2^-8 of each weight, as
// a bf16 output is rounded by 2^-8, and over many tokens less.  The exponentials are ex2.approx, off by 2^-22 or so of themselves.
//
// E4M3 caches: K goes into the products as it is, with Q as the sum of two E4M3 numbers
// (a bf16 value is one, to 2^-17 of its row's largest).  P would not be: its small values
// matter together.  So four more warps turn each tile of V into fp16, exactly, and P is
// fp16, scaled by 2^7 (f16x2_weights).  (1024 rows behind 24000 tokens, twice, 32 heads: 543 to 549 us; with K converted
// too 711: shared memory, which the conversion reads and writes as well, had 2500 cycles of work a tile.)
//
// What a row may not see is masked in S; in P V its values count 0 times.  Infinities and NaN
// among them show in the row's sums: rows whose sums are not finite are computed again key by key,
// each with its own keys only.  Behind a sequence's last token that would be common (memory
// that nothing has been written to), so there values are zeroed in shared memory.
//
// Warp roles: 0 K and V by TMA, 1 and 2 the MMAs of the two tiles, 3 Q by TMA and the
// zeroing of values behind the sequences, 4-7 and 8-11 the softmax of the two tiles, 12-15
// (E4M3) the conversion.  CTAs are persistent and every role runs ahead as far as its
// inputs allow: the next rows' first tiles arrive while the last ones are finished.
// Every wait is bounded, as in fp8_linear_tc.cu; a timeout is recorded in a word of the
// library's.
//
// Few rows behind many cached tokens (fewer CTAs' work than SMs): the cached tokens
// of each piece of work are cut into parts, whose sums a second kernel joins.
#include <cstring>

#include "paged.h"

namespace fp4moe {

namespace {

__device__ int32_t prompt_status[kStatusInts];

template <int N>
struct Const {
  static constexpr int value = N;
};

constexpr int kKeys = 128;      // cached tokens of a tile
constexpr int kPanel = kKeys * 128;  // 128 rows of 128 bytes (64 columns), 128-byte swizzle

constexpr int kSms = 152;
constexpr int kMaxItems = 32;   // pieces of work a CTA
constexpr int kMaxParts = 32;   // parts that one is cut into
constexpr int kPartTiles = 4;   // tiles of cached tokens a part has at least
constexpr int kRowsOf = 256;    // rows of a piece of work
constexpr uint64_t kLongWaits = 64;  // limit of a wait for long work, in usual ones

// A piece of work: up to two tiles of rows of one sequence and key-value head, and
// the part of their cached tokens.
struct Item {
  int64_t pos0;          // position of the first token
  int b, row0;           // sequence, first row
  uint16_t kh, tokens;   // key-value head, number of tokens
  uint8_t part, parts;
  bool ends;             // its last row is the sequence's last
};

// A piece of work that was cut: its first part, and the CTA that has it (the others follow).
struct Join {
  Item it;
  int cta;
};

struct PromptParams {
  CUtensorMap tmq, tmk, tmv;
  PagedAttn a;
  float* part;         // [grid][kRowsOf][D] sums of parts
  float2* ml;          // [grid][kRowsOf] their maxima (base 2) and sums
  Join* joins;         // [kSms] one a piece of work; parts <= 1: nothing to join
  int tile_tokens;     // tokens of one tile of rows: 128 / group
  int group_inv;       // ceil(2^16 / group)
  int split;           // whether cached tokens may be cut into parts
  int withhold;        // test knob: the first keys never arrive
  uint64_t wait_ns;
};

template <int D, bool FP8>
struct PromptCfg {
  static constexpr int kPanels = D / 64, kTile = kPanels * kPanel;  // bytes of a tile of 16-bit rows
  // bf16: K and V tiles in turn through one ring.  E4M3: K tiles as they are, raw V tiles, and
  // fp16 V tiles, each through a ring of its own.
  static constexpr int kStages = FP8 ? (D == 128 ? 2 : 4) : (D == 128 ? 4 : 8);
  static constexpr int kRaw = FP8 ? kKeys * D : 0, kKStages = FP8 ? 4 : 0, kRawStages = FP8 ? 2 : 0;
  // Q as two E4M3 tiles: over the 16-bit one, or (64: a row would lie over others') beside it
  static constexpr int kQ8 = FP8 && D == 64 ? 2 * kTile : 0;
  // outputs are staged in memory of their own, 4 KB a softmax warp, or (E4M3: no room) in Q's
  static constexpr int kStaging = FP8 ? 0 : 8 * 4096;
  static constexpr int kSmem = 2 * kTile + kStages * kTile + (kKStages + kRawStages) * kRaw + kQ8 + kStaging + 1024;
  static constexpr int kThreads = FP8 ? 512 : 384;
  // bf16: launched with 168 registers a thread, 128 x 88 + 256 x 208 = 384 x 168;
  // E4M3: with 128, 128 x 72 + 256 x 184 + 128 x 72 = 512 x 128
  static constexpr int kCtlRegs = FP8 ? 72 : 88, kSoftRegs = FP8 ? 184 : 208;
};

// ------------------------------------------------------------------ instructions
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// D += A B (kind::f16), A and B from shared memory, or A [128 x 16] from tensor memory
// (two 16-bit values a column), by the calling lane.  a, b: the low words of the
// descriptors (address and leading offset).
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;  // 8 rows in 1024 bytes, version, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) { return saddr >> 4 | (lbo >> 4) << 16; }
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, q;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
// ... of E4M3 (kind::f8f6f4, 32 columns); heads of 64: rows of 64 bytes, 64-byte swizzle.
template <int D>
__device__ __forceinline__ void tc_mma_ss_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  constexpr uint32_t kHigh = D == 128 ? kDescHigh : (512 >> 4) | 1u << 14 | 4u << 29;
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, q;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kHigh)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 db;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, q;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// After tc_wait_ld: keeps the uses of fetched values behind the wait.
template <int N>
__device__ __forceinline__ void landed(float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]),
                      "+f"(v[i + 7]));
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Shared-memory writes of this thread before tensor-core and TMA accesses that follow.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Operand formats of kind::f16: 0 fp16, 1 bf16; B of P V has its columns consecutive.
template <bool FP8>
__host__ __device__ constexpr uint32_t idesc_16(uint32_t n, bool b_rows) {
  return 1u << 4 | (FP8 ? 0u : 1u << 7 | 1u << 10) | (b_rows ? 1u << 16 : 0u) | (n >> 3) << 17 | (128u >> 4) << 24;
}

// The n lowest bits, all for n >= 32.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 16-byte piece c of a warp's staged row r: 8 rows' pieces c in different banks.
template <int ROWBYTES>
__device__ __forceinline__ uint32_t staged(int r, int c) {
  return r * ROWBYTES + ((ROWBYTES == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4);
}

// ------------------------------------------------------------------ a CTA's work
struct Work {
  Item it;
  int tiles;          // of rows
  int lo, hi, sinks;  // tokens in sight of any row: [0, sinks) and [lo, hi)
  int first, from;    // tiles of 128 of them, a list: `first` from token 0 on, then from tile `from` on
  int all, i0, n;     // the list's length, and this part's entries i0 .. i0 + n - 1
  __device__ __forceinline__ int at(int i) const { return kKeys * (i < first ? i : from + (i - first)); }
  // whether entry i has tokens behind the sequence's last one
  __device__ __forceinline__ bool edge(int i) const { return it.ends && i + 1 == all && at(i) + kKeys > hi; }
};

__device__ __forceinline__ Work work_of(const Item& it, const PagedAttn& a, int tile_tokens) {
  Work w;
  w.it = it;
  w.tiles = it.tokens > tile_tokens ? 2 : 1;
  const int64_t last = it.pos0 + it.tokens - 1;
  w.hi = it.tokens && it.pos0 < a.batch.reach && last >= 0 ? (int)min(last, (int64_t)a.batch.reach - 1) + 1 : 0;
  w.lo = w.hi > 0 && a.window > 0 ? max(0, (int)max(it.pos0, (int64_t)0) + 1 - a.window) : 0;
  w.sinks = min(a.sinks, w.hi);
  w.from = w.lo / kKeys;
  w.first = min((w.sinks + kKeys - 1) / kKeys, w.from);
  w.all = w.hi > 0 ? w.first + (w.hi + kKeys - 1) / kKeys - w.from : 0;
  w.i0 = w.all * it.part / it.parts;
  w.n = w.all * (it.part + 1) / it.parts - w.i0;
  return w;
}

// One row's query head by one warp, over the tokens of the part: D / 32 values of the row a lane,
// not yet divided by the sum l; m: the maximum (base 2).
template <int D, bool FP8>
__device__ __forceinline__ void attend_by_key(const PagedAttn& a, const Work& w, int64_t row, const Seen& seen, int h, int lane,
                                              float* o, float& m, float& l) {
  constexpr int N = D / 32;
  const int kh = w.it.kh;
  const float s1 = a.scale_log2 * (FP8 ? a.kv.k_scale[kh] : 1.f);
  float q[N];
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = bf16_to_f32(a.q[row * a.q_ld + (int64_t)h * D + N * lane + i]);
    o[i] = 0.f;
  }
  const uint8_t *kb = a.kv.k + kh * a.kv.k_head + N * lane * (FP8 ? 1 : 2),
                *vb = a.kv.v + kh * a.kv.v_head + N * lane * (FP8 ? 1 : 2);
  // (the list's entries before `first`, then the others)
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int e0 = side ? max(w.i0, w.first) : min(w.i0, w.first), e1 = side ? max(w.i0 + w.n, w.first) : min(w.i0 + w.n, w.first);
    const int j1 = e1 > e0 ? min(seen.n, w.at(e1 - 1) + kKeys) : 0;
#pragma unroll 1
    for (int j0 = w.at(e0); j0 < j1; j0 += 4) {  // four keys' loads together
      uint32_t kw[4][N / 2], vw[4][N / 2];       // (E4M3: one half of a word, two values)
      float x[4], top = -INFINITY;
      bool held[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = j0 + y, page = j < j1 && sees(seen, j) ? page_of(a.kv, a.batch, w.it.b, j) : -1;
        const int slot = j & ((1 << a.kv.page_shift) - 1);
        held[y] = page >= 0;
        const uint8_t *kp = kb + (int64_t)max(page, 0) * a.kv.k_page + slot * a.kv.k_token;
        const uint8_t *vp = vb + (int64_t)max(page, 0) * a.kv.v_page + slot * a.kv.v_token;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          kw[y][i] = vw[y][i] = 0;
          if (held[y]) {
            if constexpr (FP8) {
              kw[y][i] = *reinterpret_cast<const uint16_t*>(kp + 2 * i);
              vw[y][i] = *reinterpret_cast<const uint16_t*>(vp + 2 * i);
            } else {
              kw[y][i] = *reinterpret_cast<const uint32_t*>(kp + 4 * i);
              vw[y][i] = *reinterpret_cast<const uint32_t*>(vp + 4 * i);
            }
          }
        }
      }
      auto value = [&](uint32_t u, int i) {
        if constexpr (FP8) {
          const float4 f = e4m3x4_values(u);
          return i ? f.y : f.x;
        } else {
          return i ? bf16_hi(u) : bf16_lo(u);
        }
      };
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x[y] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) x[y] = fmaf(q[i], value(kw[y][i / 2], i & 1), x[y]);
      }
#pragma unroll
      for (int s = 16; s; s >>= 1)
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] += __shfl_xor_sync(0xffffffffu, x[y], s);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        x[y] = held[y] ? x[y] * s1 : -INFINITY;
        top = max_nan(top, x[y]);
      }
      const float now = max_nan(m, top), f = m == -INFINITY ? 0.f : exp2_approx(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] *= f;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (!held[y]) continue;
        const float e = now == -INFINITY ? 0.f : exp2_approx(x[y] - now);
        l += e;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(e, value(vw[y][i / 2], i & 1), o[i]);
      }
    }
  }
}

// A softmax warp's 32 rows, staged in shared memory, to global memory.
struct Rows {
  uint32_t stg;
  int row0, tok0;  // the first one's row of its tile, the tile's first token
  int group, group_inv, tile_tokens, tokens, lane;
  // by row: row r to dst + r * token_ld; else token k's head h to dst + k * token_ld + h * head_ld
  template <int ROWBYTES, bool BY_ROW>
  __device__ __forceinline__ void store(uint8_t* dst, int64_t token_ld, int64_t head_ld) const {
    constexpr int kLanes = ROWBYTES / 16, kAt = 32 / kLanes;
    __syncwarp();
    uint4 v[32 / kAt];
#pragma unroll
    for (int i = 0; i < 32 / kAt; ++i) v[i] = lds128(stg + staged<ROWBYTES>(i * kAt + lane / kLanes, lane % kLanes));
#pragma unroll
    for (int i = 0; i < 32 / kAt; ++i) {
      const int r = row0 + i * kAt + lane / kLanes, q = (r * group_inv) >> 16;
      if (q < tile_tokens && tok0 + q < tokens)
        *reinterpret_cast<uint4*>(dst + (BY_ROW ? r * token_ld : (tok0 + q) * token_ld + (r - q * group) * head_ld) +
                                  16 * (lane % kLanes)) = v[i];
    }
    __syncwarp();
  }
};

// N columns of this thread's row of O, times f and then vs (their product may leave the range that the output is in);
// zeros where nothing is seen (then what tensor memory holds means nothing).
template <int N = 32>
__device__ __forceinline__ void fetch_out(uint32_t taddr, float l, float f, float vs, float* o) {
#pragma unroll
  for (int x = 0; x < N; x += 32) tc_ld32(taddr + x, o + x);
  tc_wait_ld();
  landed<N>(o);
#pragma unroll
  for (int x = 0; x < N; ++x) o[x] = l == 0.f ? 0.f : o[x] * f * vs;
}

// `width` finished columns of one row from `col` on as zeros, by a warp.  (store_cols128 here had heads of 64 in E4M3 spill.)
__device__ __forceinline__ void zero_cols(const PagedOut& o, int64_t row, int col, int width, int lane) {
  const int64_t at = row * o.cols + col;
  for (int c = 8 * lane; c < width; c += 256) {
    if (o.out)
      *reinterpret_cast<uint4*>(o.out + at + c) = make_uint4(0, 0, 0, 0);
    else
      *reinterpret_cast<uint2*>(o.codes + at + c) = make_uint2(0, 0);
  }
  if (!o.out)
    for (int c = lane; c < width >> 7; c += 32) o.scales[row * (o.cols >> 7) + (col >> 7) + c] = 0.f;
}

// Pieces of a sequence whose rows are s0 .. s1 - 1.
__device__ __forceinline__ int pieces_of(const PagedBatch& bt, int b, int per, int& s0, int& end) {
  s0 = max(0, bt.starts[b]);
  end = bt.starts[b + 1];
  const int s1 = min(bt.rows, end);
  return s1 > s0 ? (s1 - s0 + per - 1) / per : 0;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(PromptCfg<D, FP8>::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = PromptCfg<D, FP8>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Item items[kMaxItems];
  __shared__ __align__(8) uint64_t bar_q, bar_q_free, bar_q16, bar_full[C::kStages], bar_empty[C::kStages], bar_s[2][2], bar_p[2][2][3],
      bar_o[2][2], bar_turn[2], bar_edge, bar_fix, bar_done, bar_raw_full[2], bar_raw_empty[2],
      bar_k_full[4], bar_k_empty[4];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, long_flag, scan_sum[C::kThreads / 32];

  const PagedAttn& a = p.a;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // Q, the ring of 16-bit tiles, (E4M3) K's ring, raw V's, Q as E4M3, or staging
  const uint32_t sq = sbase, skv = sbase + 2 * C::kTile, sk8 = skv + C::kStages * C::kTile, sraw = sk8 + C::kKStages * C::kRaw;
  const uint32_t sq8 = C::kQ8 ? sraw + C::kRawStages * C::kRaw : sq, sout = FP8 ? sq : sk8;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    mbar_init(smem_u32(&bar_q), 1);
    mbar_init(smem_u32(&bar_q_free), FP8 ? 9 : 2);
    mbar_init(smem_u32(&bar_q16), 8);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), FP8 ? 4 : 1);
      mbar_init(smem_u32(&bar_empty[s]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&bar_s[t][h]), 1);
        mbar_init(smem_u32(&bar_o[t][h]), 1);
        for (int x = 0; x < 3; ++x) mbar_init(smem_u32(&bar_p[t][h][x]), 4);
      }
      mbar_init(smem_u32(&bar_turn[t]), 1);
      mbar_init(smem_u32(&bar_raw_full[t]), 1);
      mbar_init(smem_u32(&bar_raw_empty[t]), 4);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(smem_u32(&bar_k_full[s]), 1);
      mbar_init(smem_u32(&bar_k_empty[s]), 2);
    }
    mbar_init(smem_u32(&bar_edge), 1);
    mbar_init(smem_u32(&bar_fix), 1);
    mbar_init(smem_u32(&bar_done), 2);
    abort_flag = long_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p.tmq);
    prefetch_tmap(&p.tmk);
    prefetch_tmap(&p.tmv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's items: of all pieces of work, the last of the last sequence first
  // (long causal rows before short ones), each over all heads
  int count = 0;
  {
    const int per = 2 * p.tile_tokens, B = a.batch.seqs, chunk = (B + C::kThreads - 1) / C::kThreads;
    const int b0 = min(B, tid * chunk), b1 = min(B, b0 + chunk);
    int mine = 0, s0 = 0, end = 0, len = b0 < b1 ? a.batch.lens[b0] : 0;
    for (int b = b0; b < b1; ++b) mine += pieces_of(a.batch, b, per, s0, end);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan_sum[warp] = upto;
    __syncthreads();
    int total = 0;
    upto -= mine;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) upto += scan_sum[w];
      total += scan_sum[w];
    }
    const int G = gridDim.x, pieces = total * a.kv.heads;
    const int cut = p.split && pieces > 0 ? max(1, min(kMaxParts, min(G, kSms) / pieces)) : 1;
    for (; count < kMaxItems; ++count) {
      const int v = count * G + (count & 1 ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
      if (v >= pieces * cut) break;
      const int u = v / cut, idx = total - 1 - u / a.kv.heads;
      if (upto <= idx && idx < upto + mine) {
        int b = b0, at = upto;
        if (chunk > 1) {
          for (;; ++b) {
            const int n = pieces_of(a.batch, b, per, s0, end);
            if (idx < at + n) break;
            at += n;
          }
          len = a.batch.lens[b];
        }
        Item it;
        it.b = b;
        it.kh = (uint16_t)(u % a.kv.heads);
        it.row0 = s0 + (idx - at) * per;
        it.tokens = (uint16_t)min(per, min(a.batch.rows, end) - it.row0);
        it.pos0 = (int64_t)len - end + it.row0;
        it.ends = it.row0 + it.tokens == end;
        it.part = 0;
        it.parts = 1;
        if (cut > 1) {
          it.parts = (uint8_t)max(1, min(cut, work_of(it, a, p.tile_tokens).all / kPartTiles));
          it.part = (uint8_t)(v % cut);
          if (it.part == 0) p.joins[u] = Join{it, v};
          if (it.part >= it.parts) it.part = 0, it.parts = 1, it.tokens = 0;
        }
        items[count] = it;
      }
    }
    if (p.split && tid == 0 && blockIdx.x < kSms && (cut == 1 || (int)blockIdx.x >= pieces)) p.joins[blockIdx.x] = Join{};
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  volatile int* abort_v = &abort_flag;
  auto timed_out = [&]() {  // by one lane
    if (!*abort_v) record_status(prompt_status, FP4MOE_ERR_TIMEOUT, ST_TIMEOUT);
    *abort_v = 1;
  };
  // Bounded, and longer once this CTA's softmax is at long work: rows key by key (2^24 keys a
  // row, 32 rows a warp: some 80 s), or thousands of tiles.
  volatile int* long_v = &long_flag;
  auto wait = [&](uint64_t* bar, uint32_t par) {
    if (mbar_try_wait(smem_u32(bar), par & 1u)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
      if (mbar_try_wait(smem_u32(bar), par & 1u)) return true;
      if ((i & 255u) == 0 && (*abort_v || globaltimer() - t0 > (*long_v ? kLongWaits * p.wait_ns : p.wait_ns))) return false;
    }
  };
  auto wait_w = [&](uint64_t* bar, uint32_t par) { return __all_sync(0xffffffffu, wait(bar, par)) != 0; };
  // Phases of barriers are counted over all items, ring positions too: position x is stage
  // x % kStages in its (x / kStages)-th use.
  // Tensor memory, heads of 128: S of either tile (P takes its place), O of either.  Heads of 64
  // leave room for a third S: the two tiles' entries go through the three in turn, so that a
  // tile's next S is there when its softmax has ended.  A softmax may then be two entries ahead of
  // its tile's P V: the barriers of S, P and P V are two each, used alternately.
  constexpr bool kThree = D == 64;
  auto s_at = [&](int t, int i) { return tmem + 128 * (kThree ? (2 * i + t) % 3 : t); };
  const uint32_t o_at = tmem + (kThree ? 384 : 256);
  auto side = [](uint32_t step) { return kThree ? step & 1 : 0; };
  auto turn_of = [](uint32_t step) { return kThree ? step >> 1 : step; };
  // K and V of the x-th tile:
  auto k_pos = [](uint32_t x) { return FP8 ? x : 2 * x; };
  auto v_pos = [](uint32_t x) { return FP8 ? x : 2 * x + 1; };
  constexpr uint32_t kKRing = FP8 ? C::kKStages : C::kStages;
  uint64_t *const k_full = FP8 ? bar_k_full : bar_full, *const k_empty = FP8 ? bar_k_empty : bar_empty;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kCtlRegs));
  if (warp == 0) {
    // ------------------------------------------------------------ K and V by TMA
    // a lane a page: its tokens are page_rows rows of the tile
    const int page_rows = 1 << a.kv.page_shift, boxes = kKeys >> a.kv.page_shift;
    uint32_t tiles = 0, last[2] = {0, 0};  // last: positions up to which K and V were started
    bool ok = true;
    for (int k = 0; ok && k < count; ++k) {
      const Work w = work_of(items[k], a, p.tile_tokens);
      // pages without a token in sight, and holes: past the last page, where TMA fills in zeros
      auto page_at = [&](int i) {
        int page = -1;
        if (i < w.n && lane < boxes) {
          const int j = w.at(w.i0 + i) + lane * page_rows;
          if (j < w.hi && (j + page_rows > w.lo || j < w.sinks)) page = page_of(a.kv, a.batch, w.it.b, j);
        }
        return page < 0 ? a.kv.pages : page;
      };
      int page = page_at(0);
      for (int i = 0; ok && i < w.n; ++i) {
        const int next = page_at(i + 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t pos = kv ? v_pos(tiles) : k_pos(tiles), size = kv && FP8 ? C::kRawStages : kKRing, stage = pos % size;
          uint64_t *full = kv && FP8 ? bar_raw_full : k_full, *empty = kv && FP8 ? bar_raw_empty : k_empty;
          if (!wait_w(&empty[stage], (pos / size & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[stage]);
          if (!(p.withhold && k == 0 && i == 0 && kv == 0)) {
            if (lane == 0) mbar_arrive_expect_tx(fb, FP8 ? C::kRaw : C::kTile);
            __syncwarp();
            if (lane < boxes) {
              const CUtensorMap* m = kv ? &p.tmv : &p.tmk;
              if constexpr (FP8) {
                tma_load_4d((kv ? sraw : sk8) + stage * C::kRaw + lane * page_rows * D, m, fb, 0, 0, w.it.kh, page);
              } else {
                const uint32_t dst = skv + stage * C::kTile + lane * page_rows * 128;
#pragma unroll
                for (int c = 0; c < C::kPanels; ++c) tma_load_4d(dst + c * kPanel, m, fb, 128 * c, 0, w.it.kh, page);
              }
            }
            last[kv] = pos + 1;
          }
        }
        if (ok) ++tiles;
        page = next;
      }
    }
    if (!ok && lane == 0) timed_out();
    // what was started lands before the CTA exits: the last use of every stage
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t size = kv && FP8 ? C::kRawStages : kKRing, step = FP8 ? 1 : 2;
      uint64_t* full = kv && FP8 ? bar_raw_full : k_full;
      for (uint32_t pos = last[kv] > size ? last[kv] - size : (FP8 ? 0u : (uint32_t)kv); pos < last[kv]; ++pos)
        if (pos % step == (FP8 ? 0u : (uint32_t)kv) && !(p.withhold && pos == 0 && kv == 0))
          (void)mbar_wait(smem_u32(&full[pos % size]), pos / size & 1u);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers
    // One for each tile of rows, all by one lane: the waits and commits between two runs of
    // MMAs take one issuer 700 cycles a tile, in which the other's MMAs run.  (One issuer:
    // 3700 cycles an iteration.  Where the whole warp waited and one lane issued, a wait
    // after a run of MMAs cost 1900 cycles.)
    const int t = warp - 1;
    if (elect_one()) {
      constexpr uint32_t kStep = C::kTile >> 4;
      const uint32_t dq = desc_low(FP8 ? sq8 : sq, 16), dk = desc_low(FP8 ? sk8 : skv, 16), dv = desc_low(skv, kPanel);
      const uint32_t to = o_at + D * t;
      bool ok = true;
      uint32_t tile = 0, queries = 0, edges = 0, turns = 0, done0 = 0, done1 = 0;  // done: entries of either tile before this item's
      for (int k = 0; ok && k < count; ++k) {
        const Work w = work_of(items[k], a, p.tile_tokens);
        if (w.n == 0) continue;
        const bool two = w.tiles == 2;
        if (!(ok = wait(FP8 ? &bar_q16 : &bar_q, queries))) break;
        ++queries;
        if (t >= w.tiles) {
          // Nothing to do for this tile, but in step with the other: who waits for a barrier's
          // phase has to have waited for the one before.
          mbar_arrive(smem_u32(&bar_q_free));
          tile += w.n;
          done0 += w.n;
          continue;
        }
        auto commit = [&](uint64_t* bar) {  // two arrivals, of which the other tile's issuer makes one
          tc_commit(smem_u32(bar));
          if (!two) tc_commit(smem_u32(bar));
        };
        auto k_wait = [&](int i) { return wait(&k_full[k_pos(tile + i) % kKRing], k_pos(tile + i) / kKRing); };
        auto k_free = [&](int i) { return &k_empty[k_pos(tile + i) % kKRing]; };
        // S = Q K^T of tile u and entry i
        auto scores = [&](int u, int i) {
          const uint32_t stage = k_pos(tile + i) % kKRing, qu = dq + u * kStep, s = s_at(u, i);
          if constexpr (FP8) {
            const uint32_t k0 = dk + stage * (C::kRaw >> 4);
#pragma unroll
            for (int n = 0; n < 2; ++n)  // Q's two numbers
#pragma unroll
              for (int c = 0; c < D / 32; ++c)
                tc_mma_ss_f8<D>(s, qu + ((n * kKeys * D + 32 * c) >> 4), k0 + 2 * c, idesc_f8(kKeys), n || c ? 1u : 0u);
          } else {
            const uint32_t k0 = dk + stage * kStep;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t off = ((c >> 2) * kPanel + (c & 3) * 32) >> 4;
              tc_mma_ss(s, qu + off, k0 + off, idesc_16<FP8>(kKeys, false), c ? 1u : 0u);
            }
          }
          tc_commit(smem_u32(&bar_s[u][side((u ? done1 : done0) + i)]));
        };
        // After P V of its entry i an issuer starts the S that takes that P's place: its own of
        // entry i + 1, or of three the other tile's of i + 1 (by the first issuer) or i + 2
        // (by the second; a tile alone takes every other of the three).
        const int lead = !kThree || (two && t == 0) ? 1 : 2, next = kThree && two ? 1 - t : t;
        if (!kThree || t == 0) {
          // (the other's last P V is done: its place is taken)
          if (kThree && done1 && !(ok = wait(&bar_o[1][side(done1 - 1)], turn_of(done1 - 1)))) break;
          if (!(ok = k_wait(0))) break;
          tc_fence_after();
          scores(t, 0);
          if (kThree && two) scores(1, 0), tc_commit(smem_u32(k_free(0)));
          commit(k_free(0));
          if (kThree && w.n > 1) {
            if (!(ok = k_wait(1))) break;
            tc_fence_after();
            scores(0, 1);
            commit(k_free(1));
          }
        }
        if ((!FP8 || t == 1) && w.n <= lead) tc_commit(smem_u32(&bar_q_free));  // the last scores are under way
        for (int i = 0; i < w.n; ++i) {
          const uint32_t vst = v_pos(tile + i) % C::kStages, step = (t ? done1 : done0) + i;
          if (!(ok = wait(&bar_full[vst], v_pos(tile + i) / C::kStages))) break;
          if (!FP8 && t == 0 && w.edge(w.i0 + i)) {  // warp 3 zeroes what lies behind (the other tile's turn is later)
            mbar_arrive(smem_u32(&bar_edge));
            if (!(ok = wait(&bar_fix, edges))) break;
            ++edges;
          }
          const bool more = i + lead < w.n;
          if (more && !(ok = k_wait(i + lead))) break;
          if (!(ok = wait(&bar_p[t][side(step)][0], turn_of(step)))) break;
          // Turns: the runs of the two tiles do not mix, so that one tile's softmax goes on
          // while the other's MMAs run (both fell into step otherwise: 4250 cycles an iteration).
          if (two && (t || turns) && !(ok = wait(&bar_turn[t], t ? turns : turns - 1))) break;
          tc_fence_after();
          const uint32_t v0 = dv + vst * kStep, pt = s_at(t, i);
#pragma unroll
          for (int c = 0; c < kKeys / 16; ++c) {
            if (c == 4 || c == 6) {  // 64 columns of P are there, and 32 more
              if (!(ok = wait(&bar_p[t][side(step)][c / 2 - 1], turn_of(step)))) break;
              tc_fence_after();
            }
            tc_mma_ts(to, pt + 8 * c, v0 + ((c * 2048) >> 4), idesc_16<FP8>(D, true), c ? 1u : (uint32_t)i);
          }
          if (!ok) break;
          if (kThree || i + 1 == w.n) tc_commit(smem_u32(&bar_o[t][side(step)]));
          if (more) scores(next, i + lead);  // (after P V in the tensor core's order: S takes P's place)
          if (two) mbar_arrive(smem_u32(&bar_turn[1 - t])), ++turns;
          if ((!FP8 || t == 1) && i + 1 + lead == w.n) tc_commit(smem_u32(&bar_q_free));
          commit(&bar_empty[vst]);
          if (more) commit(k_free(i + lead));
        }
        tile += w.n;
        done0 += w.n;
        if (two) done1 += w.n;
      }
      tc_commit(smem_u32(&bar_done));  // all MMAs finish before tensor memory is released
      (void)mbar_wait(smem_u32(&bar_done), 0);
      if (!ok) timed_out();
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q by TMA, values behind the sequences
    uint32_t queries = 0, tile = 0, edges = 0;
    bool ok = true;
    for (int k = 0; ok && k < count; ++k) {
      const Work w = work_of(items[k], a, p.tile_tokens);
      if (w.n == 0) continue;
      if (queries && !(ok = wait_w(&bar_q_free, (queries - 1) & 1))) break;
      if (lane == 0) {
        const int rows = a.group * p.tile_tokens;
        mbar_arrive_expect_tx(smem_u32(&bar_q), w.tiles * C::kPanels * rows * 128);
        for (int t = 0; t < w.tiles; ++t)
          for (int c = 0; c < C::kPanels; ++c)
            tma_load_3d(sq + t * C::kTile + c * kPanel, &p.tmq, smem_u32(&bar_q), 128 * c, w.it.kh * a.group,
                        w.it.row0 + t * p.tile_tokens);
      }
      __syncwarp();
      ++queries;
      if constexpr (!FP8) {
        const int i = w.i0 + w.n - 1;  // (E4M3: the conversion does it)
        if (w.edge(i)) {
          if (!(ok = wait_w(&bar_edge, edges & 1))) break;  // (the first tile's issuer has waited for the values)
          ++edges;
          const uint32_t at = skv + v_pos(tile + w.n - 1) % C::kStages * C::kTile;
          const int n = w.hi - w.at(i);
          for (int x = lane + n * 8; x < kKeys * 8; x += 32) {
#pragma unroll
            for (int c = 0; c < C::kPanels; ++c)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + c * kPanel + 16 * x), "r"(0) : "memory");
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_fix));
        }
        tile += w.n;
      }
    }
    if (!ok && lane == 0) timed_out();
    if (queries) (void)mbar_wait(smem_u32(&bar_q), (queries - 1) & 1);
    __syncwarp();
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int t = (warp - 4) >> 2, r = 32 * (warp & 3) + lane;  // tile, row of it
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, to = o_at + D * t + lanes;
    const uint32_t stg = sout + (FP8 ? t * C::kTile : t * 16384) + (warp & 3) * 4096;
    const int row_tok = (r * p.group_inv) >> 16, row_head = r - row_tok * a.group;  // r / group
    const bool row_in = r < a.group * p.tile_tokens;
    bool ok = true;
    uint32_t queries = 0, steps = 0, outs = 0;
    for (int k = 0; ok && k < count; ++k) {
      const Work w = work_of(items[k], a, p.tile_tokens);
      if (w.n == 0) {
        // Nothing in sight: zeros, a token a warp.  Not by way of shared memory: with E4M3 caches that is Q's, and the
        // next piece's Q may be on its way.  (Q is not loaded for such a piece, and no role counts it.)
        const int cols = a.group * D;
        for (int tk = t * p.tile_tokens + (warp & 3); tk < min((int)w.it.tokens, (t + 1) * p.tile_tokens); tk += 4)
          zero_cols(a.out, w.it.row0 + tk, w.it.kh * cols, cols, lane);
        __syncwarp();
        continue;
      }
      if (w.n > 4096) *long_v = 1;
      const int tok = t * p.tile_tokens + row_tok;
      const bool mine = row_in && tok < w.it.tokens;
      Seen seen = {0, 0, 1 << 30};  // a row that is not stored is not masked
      if (mine) seen = seen_from(w.it.pos0 + tok, a.batch.reach, a.window, a.sinks);
      // what all rows of the warp see
      const int all_n = __reduce_min_sync(0xffffffffu, seen.n), all_lo = __reduce_max_sync(0xffffffffu, seen.lo),
                all_sinks = __reduce_min_sync(0xffffffffu, mine ? seen.sinks : 1 << 30);
      float scale = a.scale_log2;
      bool spoilt = false;
      if constexpr (FP8) {
        // Q as the sum of two E4M3 numbers, for products with the cache's codes as they are.
        // Scaled by the power of two that brings a row's largest magnitude to 128 .. 256, the 8 bits
        // of a bf16 value are the first number's 4 and a remainder of 4: exact down to 2^-9 of
        // the largest, and below off by half of E4M3's smallest step, 2^-10: 2^-17 of the largest at most.
        // (A largest one below 2^-119 comes to less than 128.)
        if (!(ok = wait_w(&bar_q, queries & 1))) break;
        if (t < w.tiles) {
          uint4 q[D / 8];
          float amax = 0.f;
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            q[x] = lds128(sq + t * C::kTile + (x >> 3) * kPanel + r * 128 + (((x & 7) ^ (r & 7)) << 4));
#pragma unroll
            for (uint32_t y : {q[x].x, q[x].y, q[x].z, q[x].w}) amax = max_nan(amax, max_nan(fabsf(bf16_lo(y)), fabsf(bf16_hi(y))));
          }
          const int e = (int)(__float_as_uint(amax) >> 23 & 255u);
          const int x2 = max(e - 134, -126);  // (both powers are normal numbers)
          const float down = __uint_as_float((uint32_t)(127 - x2) << 23);
          scale *= __uint_as_float((uint32_t)(127 + x2) << 23) * a.kv.k_scale[w.it.kh];
          spoilt = e == 255;  // (infinities saturate: such a row is computed key by key if it sees anything)
          const uint32_t to_q = sq8 + t * C::kTile + r * D, swz = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint4& v = q[2 * x + (y >> 1)];
              const uint32_t u0 = y & 1 ? v.z : v.x, u1 = y & 1 ? v.w : v.y;
              const float v0 = bf16_lo(u0) * down, v1 = bf16_hi(u0) * down, v2 = bf16_lo(u1) * down, v3 = bf16_hi(u1) * down;
              hi[y] = e4m3x4(v0, v1, v2, v3);
              const float4 f = e4m3x4_values(hi[y]);
              lo[y] = e4m3x4(v0 - f.x, v1 - f.y, v2 - f.z, v3 - f.w);
            }
            sts128(to_q + ((x ^ swz) << 4), hi[0], hi[1], hi[2], hi[3]);
            sts128(to_q + kKeys * D + ((x ^ swz) << 4), lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_q16));
      }
      scale = fmaxf(scale, 1.17549435e-38f);  // (a scale of 0: masked scores stay -inf)
      const float grow = fminf(8.f / scale, 3.0e38f);  // (finite: a first maximum is always taken)
      constexpr float kUp = FP8 ? 7.f : 0.f;  // weights, which may grow to 2^8, are scaled by 2^kUp (f16x2_weights)
      float m = -INFINITY, l = 0.f;
      for (int i = 0; t < w.tiles && i < w.n; ++i, ++steps) {
        const int j0 = w.at(w.i0 + i);
        // holes: a lane a group of 16 tokens
        bool held = true;
        if (lane < kKeys / kPageStep) {
          const int j = j0 + kPageStep * lane;
          held = j >= a.batch.reach || page_of(a.kv, a.batch, w.it.b, j) >= 0;
        }
        if (!(ok = wait_w(&bar_s[t][side(steps)], turn_of(steps)))) break;
        tc_fence_after();
        const uint32_t ts = s_at(t, i) + lanes;
        const unsigned holes = ~__ballot_sync(0xffffffffu, held);
        if (holes || j0 + kKeys > all_n || (j0 < all_lo && j0 + kKeys > all_sinks)) {
          // Masked in place, 32 columns at a time, a bit a column.  (Over all columns in registers: code
          // that is long and rare, 840 cycles more a tile.)
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            const int j = j0 + 32 * x;
            uint32_t v = below(seen.n - j) & (~below(seen.lo - j) | below(seen.sinks - j));
            if (holes >> (2 * x) & 1u) v &= 0xFFFF0000u;
            if (holes >> (2 * x) & 2u) v &= 0x0000FFFFu;
            if (__all_sync(0xffffffffu, v == ~0u)) continue;
            float f[32];
            uint32_t u[32];
            tc_ld32(ts + 32 * x, f);
            tc_wait_ld();
            landed<32>(f);
#pragma unroll
            for (int c = 0; c < 32; ++c) u[c] = v & (1u << c) ? __float_as_uint(f[c]) : 0xFF800000u;
            tc_st32(ts + 32 * x, u);
          }
          tc_wait_st();
        }
        float s[kKeys];
        tc_ld32(ts, s);
        tc_ld32(ts + 32, s + 32);
        tc_wait_ld();
        landed<64>(s);
        tc_ld32(ts + 64, s + 64);
        tc_ld32(ts + 96, s + 96);
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x] = max3(top[x], s[c + x], s[c + 4 + x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) top[x] = fmaxf(top[x], s[60 + x]);
        tc_wait_ld();
        landed<64>(s + 64);
#pragma unroll
        for (int c = 64; c < kKeys; c += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x] = max3(top[x], s[c + x], s[c + 4 + x]);
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        if (__any_sync(0xffffffffu, mx > m + grow)) {
          const float now = mx > m + grow ? mx : m, f = m == -INFINITY ? 0.f : exp2_approx((m - now) * scale);
          const float f1 = now == m ? 1.f : f;
          m = now;
          l *= f1;
          if (i > 0) {  // (S came after the last P V, but of three)
            if (kThree) {
              if (!(ok = wait_w(&bar_o[t][side(steps - 1)], turn_of(steps - 1)))) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tc_ld32(to + 32 * c, o);
              tc_wait_ld();
              landed<32>(o);
              uint32_t u[32];
#pragma unroll
              for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(o[x] * f1);
              tc_st32(to + 32 * c, u);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : kUp - m * scale;
        const uint64_t sc2 = pack2(scale, scale), ba2 = pack2(base, base);
        uint64_t sum[2] = {0, 0};
        uint32_t pk[32];
        auto weights = [&](auto from, auto to_) {  // pairs of columns
#pragma unroll
          for (int c = decltype(from)::value; c < decltype(to_)::value; ++c) {
            float x, y;
            unpack2(fma2(pack2(s[2 * c], s[2 * c + 1]), sc2, ba2), x, y);
            x = exp2_approx(x), y = exp2_approx(y);
            sum[c & 1] = add2(sum[c & 1], pack2(x, y));
            pk[c & 31] = FP8 ? f16x2_weights(x, y) : bf16x2_rn(x, y);
          }
        };
        auto ready = [&](int half) {
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_p[t][side(steps)][half]));
        };
        // P V starts while the second half's weights are computed
        weights(Const<0>{}, Const<32>{});
        tc_st32(ts, pk);
        weights(Const<32>{}, Const<40>{});
        ready(0);
        weights(Const<40>{}, Const<48>{});
        tc_st16(ts + 32, pk);
        weights(Const<48>{}, Const<52>{});
        ready(1);
        weights(Const<52>{}, Const<64>{});
        tc_st16(ts + 48, pk + 16);
        float x, y;
        unpack2(add2(sum[0], sum[1]), x, y);
        l += x + y;
        ready(2);
      }
      if (!ok) break;
      if (t < w.tiles && !(ok = wait_w(&bar_o[t][side(steps - 1)], kThree ? turn_of(steps - 1) : outs++))) break;
      ++queries;
      tc_fence_after();
      if (t < w.tiles) {
        // rows rr of the warp: where they go
        const bool parts = w.it.parts > 1;
        const float f = parts ? 1.f : l == 0.f ? 0.f : 1.f / l, vs = FP8 && !parts ? a.kv.v_scale[w.it.kh] : 1.f;
        // (opaque, so that what depends on the lane alone is not kept in registers over all items)
        int ln = lane;
        asm volatile("" : "+r"(ln));
        const Rows to_rows = {stg, 32 * (warp & 3), t * p.tile_tokens, a.group, p.group_inv, p.tile_tokens, (int)w.it.tokens, ln};
        const int64_t part_row = (int64_t)blockIdx.x * kRowsOf + 128 * t;
        // Infinities and NaN of V in places that a row does not see are in its sums too (0 * NaN).  (Where
        // l is NaN, all the row's outputs are.)
        float most[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          fetch_out(to + 32 * c, l, f, vs, o);
#pragma unroll
          for (int x = 0; x < 32; ++x) most[x & 3] = max_nan(most[x & 3], fabsf(o[x]));
        }
        float amax = max_nan(max_nan(most[0], most[1]), max_nan(most[2], most[3]));
        const bool by_key =
            __any_sync(0xffffffffu, mine && ((l == l && !(amax <= 3.4028235e38f)) || (spoilt && m != -INFINITY)));
        if (by_key) *long_v = 1;
        if (!by_key) {
          // through shared memory, so that stores cover whole rows (a row a lane: 4000 cycles)
          if (parts) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              fetch_out(to + 32 * c, l, f, vs, o);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                sts128(stg + staged<128>(ln, x), __float_as_uint(o[4 * x]), __float_as_uint(o[4 * x + 1]),
                       __float_as_uint(o[4 * x + 2]), __float_as_uint(o[4 * x + 3]));
              to_rows.store<128, true>(reinterpret_cast<uint8_t*>(p.part + part_row * D + 32 * c), 4 * D, 0);
            }
            if (mine) p.ml[part_row + r] = make_float2(m == -INFINITY ? m : m * scale - kUp, l);
          } else if (a.out.out) {
            uint8_t* dst = reinterpret_cast<uint8_t*>(a.out.out + (int64_t)w.it.row0 * a.out.cols + (int64_t)w.it.kh * a.group * D);
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              float o[64];
              fetch_out<64>(to + 64 * c, l, f, vs, o);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                sts128(stg + staged<128>(ln, x), bf16x2_rn(o[8 * x], o[8 * x + 1]), bf16x2_rn(o[8 * x + 2], o[8 * x + 3]),
                       bf16x2_rn(o[8 * x + 4], o[8 * x + 5]), bf16x2_rn(o[8 * x + 6], o[8 * x + 7]));
              to_rows.store<128, false>(dst + 128 * c, 2 * (int64_t)a.out.cols, 2 * D);
            }
          } else {
            // (heads of 64: rows 2i and 2i + 1 are the halves of a block)
            if constexpr (D == 64) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const float sc = e4m3_scale(amax), rc = __fdiv_rn(1.f, sc);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              fetch_out(to + 32 * c, l, f, vs, o);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t q[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const float* v = o + 16 * x + 4 * y;
                  q[y] = e4m3x4(e4m3_scaled(v[0], sc, rc), e4m3_scaled(v[1], sc, rc), e4m3_scaled(v[2], sc, rc),
                                e4m3_scaled(v[3], sc, rc));
                }
                sts128(stg + staged<D>(ln, 2 * c + x), q[0], q[1], q[2], q[3]);
              }
            }
            to_rows.store<D, false>(a.out.codes + (int64_t)w.it.row0 * a.out.cols + (int64_t)w.it.kh * a.group * D, a.out.cols, D);
            if (mine && (D == 128 || (r & 1) == 0))
              a.out.scales[(int64_t)(w.it.row0 + tok) * (a.out.cols >> 7) + (((w.it.kh * a.group + row_head) * D) >> 7)] = sc;
          }
        } else {
          // 128 columns at a time where they share a scale, else a head
          const int heads = D == 64 && a.out.codes && !parts ? 2 : 1;
#pragma unroll 1
          for (int i = 0; i < 32; i += heads) {
            const int rr = 32 * (warp & 3) + i, q = (rr * p.group_inv) >> 16, tk = t * p.tile_tokens + q;
            const int h = w.it.kh * a.group + rr - q * a.group;
            if (rr >= a.group * p.tile_tokens || tk >= w.it.tokens) break;
            const Seen sn = seen_from(w.it.pos0 + tk, a.batch.reach, a.window, a.sinks);
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 1
            for (int x = 0; x < heads; ++x) {
              float o[D / 32], km, kl;
              attend_by_key<D, FP8>(a, w, w.it.row0 + tk, sn, h + x, lane, o, km, kl);
              const float vs = parts ? 1.f : kl == 0.f ? 0.f : (FP8 ? a.kv.v_scale[w.it.kh] : 1.f) / kl;
              if (parts && lane == 0) p.ml[part_row + rr] = make_float2(km, kl);
              if constexpr (D == 128) {
                v = make_float4(o[0] * vs, o[1] * vs, o[2] * vs, o[3] * vs);
              } else {
                const int src = 2 * (lane & 15);
                const float4 y = make_float4(__shfl_sync(0xffffffffu, o[0] * vs, src), __shfl_sync(0xffffffffu, o[1] * vs, src),
                                             __shfl_sync(0xffffffffu, o[0] * vs, src + 1), __shfl_sync(0xffffffffu, o[1] * vs, src + 1));
                if ((lane >> 4) == x) v = y;
              }
            }
            if (!parts) {
              store_cols128(a.out, w.it.row0 + tk, h * D, heads * D, lane, v);
            } else {
              if (4 * lane < D) *reinterpret_cast<float4*>(p.part + (part_row + rr) * D + 4 * lane) = v;
            }
          }
        }
      }
      if constexpr (FP8) {
        fence_async_smem();  // (staged rows were written where TMA writes the next Q)
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_q_free));
      }
    }
    if (!ok && lane == 0) timed_out();
    __syncwarp();
  } else if constexpr (FP8) {
    // ------------------------------------------------------------ E4M3 to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(72));
    constexpr int kPieces = D / 16;  // 16-code pieces of a token
    int stage = 0, raw = 0;
    uint32_t phase = 0, raw_phase = 0;
    bool ok = true;
    for (int k = 0; ok && k < count; ++k) {
      const Work w = work_of(items[k], a, p.tile_tokens);
      for (int i = 0; i < w.n; ++i) {
        const int j0 = w.at(w.i0 + i);
        const bool v_edge = w.edge(w.i0 + i);
        if (!(ok = wait_w(&bar_raw_full[raw], raw_phase)) || !(ok = wait_w(&bar_empty[stage], phase ^ 1u))) break;
        const uint32_t src = sraw + raw * C::kRaw, dst = skv + stage * C::kTile;
#pragma unroll 4
        for (int x = tid - 384; x < kKeys * kPieces; x += 128) {
          const int row = x / kPieces, c = x % kPieces;
          uint4 q = lds128(src + 16 * x);
          uint32_t f[8];
          if (v_edge && j0 + row >= w.hi) q = make_uint4(0, 0, 0, 0);
          int y = 0;
#pragma unroll
          for (uint32_t z : {q.x, q.y, q.z, q.w}) {
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                : "=r"(f[2 * y]), "=r"(f[2 * y + 1])
                : "r"(z));
            ++y;
          }
          const uint32_t at = dst + (c >> 2) * kPanel + row * 128;
          sts128(at + (((2 * (c & 3)) ^ (row & 7)) << 4), f[0], f[1], f[2], f[3]);
          sts128(at + (((2 * (c & 3) + 1) ^ (row & 7)) << 4), f[4], f[5], f[6], f[7]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bar_full[stage]));
          mbar_arrive(smem_u32(&bar_raw_empty[raw]));
        }
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        if (++raw == C::kRawStages) { raw = 0; raw_phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) timed_out();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the pieces of work that were cut: a warp a row's head (two of 64
// where they share a scale).
template <int D, bool FP8>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ PromptParams p) {
  pdl_wait();
  pdl_trigger();
  const PagedAttn& a = p.a;
  const Join jn = p.joins[blockIdx.x];
  const Item& it = jn.it;
  if (it.parts <= 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = D == 64 && a.out.codes ? 2 : 1;
  const int r = 8 * blockIdx.y + warp, rr = r & 127, q = (rr * p.group_inv) >> 16, tok = (r >> 7) * p.tile_tokens + q;
  if (rr >= a.group * p.tile_tokens || tok >= it.tokens || (heads == 2 && (rr & 1))) return;
  const int own = heads == 2 ? lane >> 4 : 0, col = (4 * lane) % D;
  const int64_t at = (int64_t)jn.cta * kRowsOf + r + own;
  float4 v = make_float4(0, 0, 0, 0);
  float top = -INFINITY, sum = 0.f;
  for (int i0 = 0; i0 < it.parts; i0 += 8) {  // eight parts' loads together
    float4 x[8];
    float2 ml[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i < it.parts) {
        ml[i] = p.ml[at + (int64_t)(i0 + i) * kRowsOf];
        x[i] = *reinterpret_cast<const float4*>(p.part + (at + (int64_t)(i0 + i) * kRowsOf) * D + col);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ml[i].x == -INFINITY) continue;
      const float now = max_nan(top, ml[i].x), f = top == -INFINITY ? 0.f : exp2_approx(top - now), e = exp2_approx(ml[i].x - now);
      v = make_float4(v.x * f + x[i].x * e, v.y * f + x[i].y * e, v.z * f + x[i].z * e, v.w * f + x[i].w * e);
      sum = sum * f + ml[i].y * e;
      top = now;
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum, vs = FP8 ? a.kv.v_scale[it.kh] : 1.f;
  store_cols128(a.out, it.row0 + tok, (it.kh * a.group + rr - q * a.group) * D, heads * D, lane,
                make_float4(v.x * f * vs, v.y * f * vs, v.z * f * vs, v.w * f * vs));
}

template <int D, bool FP8>
cudaError_t launch(const PagedAttn& a, void* ws, const PromptKnobs& knobs, cudaStream_t s) {
  using C = PromptCfg<D, FP8>;
  PromptParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.tile_tokens = 128 / a.group;
  p.group_inv = (65536 + a.group - 1) / a.group;
  p.wait_ns = knobs.wait_ns ? knobs.wait_ns : kWaitLimitNs;
  p.withhold = knobs.withhold;
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.part = reinterpret_cast<float*>(at);
  at += (size_t)kSms * kRowsOf * D * 4;
  p.ml = reinterpret_cast<float2*>(at);
  at += (size_t)kSms * kRowsOf * 8;
  p.joins = reinterpret_cast<Join*>(at);
  const int size = FP8 ? 1 : 2, page = 1 << a.kv.page_shift;
  auto map_kv = [&](CUtensorMap* m, const uint8_t* base, int64_t ps, int64_t hs, int64_t ts) {
    const uint64_t dims[4] = {(uint64_t)(D * size), (uint64_t)page, (uint64_t)a.kv.heads, (uint64_t)a.kv.pages};
    // (a dimension of one is never stepped along)
    const uint64_t strides[3] = {(uint64_t)ts, (uint64_t)(hs ? hs : 16), (uint64_t)(ps ? ps : 16)};
    const uint32_t box[4] = {FP8 ? (uint32_t)D : 128u, (uint32_t)page, 1, 1};
    return encode_tmap_u8_swizzled(m, base, 4, dims, strides, box, m == &p.tmv && FP8 ? 0 : (int)box[0]);
  };
  const uint64_t qd[3] = {(uint64_t)D * 2, (uint64_t)a.q_heads, (uint64_t)a.batch.rows};
  const uint64_t qs[2] = {(uint64_t)D * 2, (uint64_t)a.q_ld * 2};
  const uint32_t qb[3] = {128, (uint32_t)a.group, (uint32_t)p.tile_tokens};
  if (!encode_tmap_u8(&p.tmq, a.q, 3, qd, qs, qb, true) || !map_kv(&p.tmk, a.kv.k, a.kv.k_page, a.kv.k_head, a.kv.k_token) ||
      !map_kv(&p.tmv, a.kv.v, a.kv.v_page, a.kv.v_head, a.kv.v_token))
    return cudaErrorInvalidValue;
  static bool attr_set[64] = {};
  if (cudaError_t e = allow_smem(prompt_kernel<D, FP8>, C::kSmem, attr_set)) return e;
  // Pieces of work: `most` at most.
  const int64_t per = 2 * p.tile_tokens;
  const int64_t most = (a.batch.rows / per + std::min(a.batch.seqs, a.batch.rows)) * a.kv.heads;
  p.split = attn_prompt_needs_workspace(a);
  const int64_t grid = std::max(p.split ? kSms : std::min(most, (int64_t)kSms), (most + kMaxItems - 1) / kMaxItems);
  if (cudaError_t e = launch_pdl(prompt_kernel<D, FP8>, dim3((unsigned)grid), dim3(C::kThreads), C::kSmem, s, p)) return e;
  const unsigned joins = (unsigned)std::min(most, (int64_t)kSms);  // (a grid of kSms: 3.5 us more to find nothing)
  return p.split ? launch_pdl(prompt_join_kernel<D, FP8>, dim3(joins, kRowsOf / 8), dim3(256), 0, s, p) : cudaSuccess;
}

}  // namespace

// Whether cached tokens may be cut into parts: few rows (where all belong to a sequence,
// they make half as many pieces of work as there are SMs or fewer) and room for two parts.
bool attn_prompt_needs_workspace(const PagedAttn& a) {
  const int64_t per = 2 * (128 / a.group);
  return 2 * ((a.batch.rows + per - 1) / per * a.kv.heads) <= kSms && a.batch.reach >= 2 * kPartTiles * kKeys;
}

size_t attn_prompt_workspace(int head_dim) { return (size_t)kSms * (kRowsOf * (4 * head_dim + 8) + sizeof(Join)); }

cudaError_t launch_attn_prompt(const PagedAttn& a, int head_dim, bool fp8, void* ws, const PromptKnobs& knobs, cudaStream_t s) {
  if (head_dim == 64) return fp8 ? launch<64, true>(a, ws, knobs, s) : launch<64, false>(a, ws, knobs, s);
  return fp8 ? launch<128, true>(a, ws, knobs, s) : launch<128, false>(a, ws, knobs, s);
}

cudaError_t attn_prompt_status_word(int32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), prompt_status);
}

}  // namespace fp4moe
