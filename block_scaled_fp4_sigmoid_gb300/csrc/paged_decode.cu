// Attention of one new token a sequence over the paged cache.
//
// What bounds it: the cache's bytes, each read once (4 bytes of bf16 a head
// value against 4 operations a query head).  So the work is cut by bytes and
// not by sequence: the groups of 16 tokens that all sequences see, over all
// key-value heads, are one list, and every CTA takes an equal run of it, whatever the
// lengths.  A sequence's head that lies in several runs leaves partial sums in
// the workspace, which a second kernel joins.  Short caches go without a plan, a
// workspace and a second kernel: a CTA, or a cluster of them, a head.
//
// In a CTA each warp streams its own groups of 16 tokens through its own ring in
// shared memory (cp.async: no barrier between warps).  Tokens are the rows of the
// products S^T = K Q^T and O^T = V^T P^T (mma.sync: the tensor cores are far from busy,
// and operands come straight from the ring), the queries that share a key-value
// head, 8 or 16, their columns; running maximum and sum of the softmax stay in
// registers and the warps' sums are joined in shared memory when the head changes.
// Weights are rounded to the operands' type, bf16 (2^-8 of each, as a bf16 output is rounded by 2^-8, and over many
// tokens less) or, for E4M3 caches, fp16 (f16x2_weights; q too, below); the sums have them unrounded.  The exponentials are
// ex2.approx, off by 2^-22 or so of themselves.
// (With the queries as the 16 rows, a group of 4 or 8 took twice the products, twice the
// exponentials and twice the registers: 64 sequences of up to 16000, E4M3, 177 us, now 168.)
#include "paged.h"

namespace fp4moe {

namespace {

constexpr int kWarps = 4, kRows = 16;  // kRows: query heads that a CTA takes at most
constexpr int kMinRun = 4 * kWarps;    // units that a CTA takes at least
constexpr int kMaxCluster = 8;
constexpr int kClusterValues = 1 << 18;  // values of K that a CTA of decode_cluster_kernel may have

struct DecodeParams {
  PagedAttn a;
  int hgroups;   // groups of up to 16 query heads a key-value head
  int cluster;   // CTAs a sequence's head (decode_cluster_kernel)
  float* part;   // [grid][2][kRows][D] sums of the runs' first and last heads, where others go on with them
  float2* ml;    // [grid][2][kRows] their maxima (base 2) and sums
  int4* joins;   // what goes on in other runs than it begins in: {sequence, head group, runs, first run}; by
                 // segment (sequence and head group) where `by_segment`, else by the run that it begins in
  int by_segment;
};

// NT: columns of 8 query heads; CL: decode_cluster_kernel; W: warps of a CTA.
template <int D, bool FP8, int NT, bool CL, int W = kWarps>
struct DecCfg {
  static constexpr int kW = W;
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2), kTile = kPageStep * kRowBytes;  // 16 tokens of K or V
  // Groups of 16 tokens of a warp's step: of E4M3 two, whose products do not wait for one
  // another (64 sequences of up to 16000, 8 heads: 168 us, one group 173).
  static constexpr int kGroups = FP8 ? 2 : 1, kStage = kGroups * 2 * kTile;
  // CTAs an SM, as registers allow, and stages of a warp's ring: 192 KB of rings an SM
  // together.  More CTAs hide each other's starts and ends, longer rings run more steadily:
  // heads of 128 in E4M3 run 168 us with three CTAs of two stages and 179 with two of three at 64
  // sequences of up to 16000; in bf16 98 us with two CTAs of three stages and 101 with three of two at
  // 38 sequences of 4095, but 32 and 26 at 256 of 100; of 64, four of three are best at both (84 us
  // at 64 sequences of 4095; three of four 106).
  static constexpr int kFours = NT == 2 ? 2 : kRowBytes == 256 ? (CL ? 3 : 2) : D == 128 ? 3 : 4, kCtas = kFours * kWarps / W;
  static constexpr int kStages = D == 64 ? 3 : kFours == 2 ? 3 : 2;
  static constexpr int kRing = W * kStages * kStage;
  static constexpr int kHeads = 8 * NT, kJoinLd = D + 4;  // (a row's padding: lanes write different banks)
  static constexpr int kJoin = W * kHeads * kJoinLd * 4;
  static constexpr int kSmem = kRing > kJoin + kHeads * D * 4 ? kRing : kJoin + kHeads * D * 4;
};

// 16-byte piece c of row r, so that 8 rows' pieces c, and two rows' 4 consecutive
// ones, lie in different banks.
template <int ROWBYTES>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if constexpr (ROWBYTES == 64)
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return r * ROWBYTES + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// d += A (16 x 16) . B (16 x 8); with lane = 4 g + t: a0, a2 from row g, a1, a3 from
// row g + 8, columns 2t, 2t + 1 (a0, a1) and 2t + 8, 2t + 9; b0, b1 those rows of
// column g; d0, d1 are row g and columns 2t, 2t + 1, d2, d3 the same of row g + 8.
template <bool F16>
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// fp16 pairs of the two low and the two high codes of a word.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The transpose of an 8 x 8 matrix of 16-bit values in a warp's registers.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The groups of 16 tokens that sequence b's new token sees, as a list: `first` of them
// from token 0 on (the sinks'), the others from group `from` on.
struct Groups {
  Seen seen;
  int first, from, n;
  __device__ __forceinline__ int at(int i) const { return i < first ? i : from + (i - first); }
  // whether all 16 tokens from j on are seen
  __device__ __forceinline__ bool whole(int j) const {
    return j + kPageStep <= seen.n && (j >= seen.lo || j + kPageStep <= seen.sinks);
  }
};
__device__ __forceinline__ Groups groups_of(const PagedAttn& a, int b) {
  Groups g;
  g.seen = seen_from((int64_t)a.batch.lens[b] - 1, a.batch.reach, a.window, a.sinks);
  g.from = g.seen.lo / kPageStep;
  g.first = min((g.seen.sinks + kPageStep - 1) / kPageStep, g.from);
  g.n = g.first + (g.seen.n + kPageStep - 1) / kPageStep - g.from;
  return g;
}

// One key-value head's run of groups [g0, g1) through a warp's ring.
template <typename C>
struct Stream {
  static constexpr int kPieces = C::kRowBytes / 16, kRowsAt = 32 / kPieces;  // 16-byte pieces of a row; rows of 32 pieces
  const PagedKv& kv;
  const Groups& gr;
  const int32_t* pages;             // the sequence's row of the table
  const int lane, g1;
  const uint32_t ring, at0;         // at0: where this lane's first piece goes
  const uint8_t *kbase, *vbase;     // the head's, at this lane's first piece of a group
  int next, next_page[C::kGroups];  // the next groups to fetch and their pages (or holes)
  unsigned fetched;                 // a bit for each group of each fetch, the last one's lowest: not a hole

  __device__ __forceinline__ Stream(const PagedAttn& a, const Groups& gr_, int b, int kh, int lane_, int warp, int g0, int g1_,
                                    uint32_t ring_)
      : kv(a.kv), gr(gr_), pages(a.batch.table + b * a.batch.table_ld), lane(lane_), g1(g1_), ring(ring_),
        at0(piece_at<C::kRowBytes>(lane_ / kPieces, lane_ % kPieces)) {
    kbase = kv.k + kh * kv.k_head + (lane / kPieces) * kv.k_token + 16 * (lane % kPieces);
    vbase = kv.v + kh * kv.v_head + (lane / kPieces) * kv.v_token + 16 * (lane % kPieces);
    next = g0 + warp * C::kGroups;
    fetched = 0;
    look();
  }
  __device__ __forceinline__ void look() {
#pragma unroll
    for (int g = 0; g < C::kGroups; ++g) {
      next_page[g] = -1;
      if (next + g < g1) {
        const int page = pages[gr.at(next + g) * kPageStep >> kv.page_shift];
        if ((unsigned)page < (unsigned)kv.pages) next_page[g] = page;
      }
    }
  }
  // Starts the next groups on their way into a stage (nothing for a hole); the pages after
  // them are looked up meanwhile.
  __device__ __forceinline__ void fetch(int stage) {
#pragma unroll
    for (int g = 0; g < C::kGroups; ++g) {
      const int page = next_page[g];
      if (page >= 0) {
        const int j0 = gr.at(next + g) * kPageStep, row0 = j0 & ((1 << kv.page_shift) - 1);
        const uint8_t* ks = kbase + page * kv.k_page + row0 * kv.k_token;
        const uint8_t* vs = vbase + page * kv.v_page + row0 * kv.v_token;
        const uint32_t dst = ring + (stage * C::kGroups + g) * 2 * C::kTile + at0;
        const bool whole = gr.whole(j0);
#pragma unroll
        for (int i = 0; i < kPageStep / kRowsAt; ++i) {
          // (rows kRowsAt apart: the swizzle's bits of the one over those of the other)
          const uint32_t to = (dst ^ (piece_at<C::kRowBytes>(i * kRowsAt, 0) & (C::kRowBytes - 1) & 0x70)) + i * kRowsAt * C::kRowBytes;
          // tokens that are not seen come as zeros: what they hold is never read
          const bool in = whole || sees(gr.seen, j0 + i * kRowsAt + lane / kPieces);
          cp_async16(to, in ? ks : kbase, in);
          cp_async16(to + C::kTile, in ? vs : vbase, in);
          ks += kRowsAt * kv.k_token;
          vs += kRowsAt * kv.v_token;
        }
      }
      fetched = fetched << 1 | (page >= 0 ? 1u : 0u);
    }
    cp_commit();
    next += C::kW * C::kGroups;
    look();
  }
};

// The joined sums of a CTA's run of one head, a row's 4 columns a lane.
struct Joined {
  float4 v;
  float top, sum;  // the row's maximum (base 2) and sum
  __device__ __forceinline__ void add(const float4& x, float2 ml) {
    if (ml.x == -INFINITY) return;
    const float now = max_nan(top, ml.x), f = top == -INFINITY ? 0.f : exp2_approx(top - now), e = exp2_approx(ml.x - now);
    v = make_float4(v.x * f + x.x * e, v.y * f + x.y * e, v.z * f + x.z * e, v.w * f + x.w * e);
    sum = sum * f + ml.y * e;
    top = now;
  }
  // the output, v_scale included
  __device__ __forceinline__ float4 out(float v_scale) const {
    const float f = sum == 0.f ? 0.f : v_scale / sum;
    return make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
};

// The groups [i0, i1) of sequence b for the nq query heads from qh on, by the CTA's
// warps; each warp's blocks of 128 columns (a head of 128, two of 64) of the result go to
// done(first row, row, column, Joined).  The ring is free again after a barrier.
template <int D, bool FP8, int NT, bool CL, int W, typename F>
__device__ __forceinline__ void attend(const PagedAttn& a, const Groups& gr, int b, int kh, int qh, int nq, int i0, int i1,
                                       uint8_t* smem, float2 (&ml)[W][kRows], F done) {
  using C = DecCfg<D, FP8, NT, CL, W>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  Stream<C> st(a, gr, b, kh, lane, warp, i0, i1, ring);
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) st.fetch(s);

  // queries: column g of the B operands; qs: factors of this lane's columns 2t and 2t + 1
  uint32_t qf[NT][D / 16][2];
  float qs[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint16_t* q0 = a.q + b * a.q_ld + (int64_t)(qh + 8 * n + g) * D;
    const bool in = 8 * n + g < nq;
    qs[n][0] = qs[n][1] = a.scale_log2;
    if constexpr (!FP8) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) qf[n][s][i] = in ? *reinterpret_cast<const uint32_t*>(q0 + 16 * s + 8 * i + 2 * t) : 0u;
    } else {
      // fp16 like the cache's values, scaled by the power of two that brings the row's
      // largest magnitude to 1 .. 2: what that loses is below 2^-24 of it
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const int at = 16 * (t + 4 * (s >> 2)) + 4 * (s & 3);  // this lane's 4 columns of step s
        uint2 w = make_uint2(0, 0);
        if (in) w = *reinterpret_cast<const uint2*>(q0 + at);
        qf[n][s][0] = w.x, qf[n][s][1] = w.y;
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(w.x)), fabsf(bf16_hi(w.x))), fmaxf(fabsf(bf16_lo(w.y)), fabsf(bf16_hi(w.y)))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // (infinities stay, and nothing beside them becomes one; both powers are normal numbers)
      const int k = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
      const float down = __uint_as_float((uint32_t)(127 - k) << 23), up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
      for (int i = 0; i < 2; ++i) qs[n][i] *= __shfl_sync(0xffffffffu, up, 4 * (2 * t + i)) * a.kv.k_scale[kh];
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) qf[n][s][i] = f16x2_rn(bf16_lo(qf[n][s][i]) * down, bf16_hi(qf[n][s][i]) * down);
    }
  }

  // o[c]: 16 columns of O; elements 0, 1 are column g (E4M3: 2g) of heads 2t and 2t + 1, elements 2, 3
  // column g + 8 (2g + 1)
  float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[n][c][0] = o[n][c][1] = o[n][c][2] = o[n][c][3] = 0.f;
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
  constexpr float kUp = FP8 ? 15.f : 0.f, kDown = FP8 ? 0x1p-15f : 1.f;  // weights are scaled by 2^kUp (f16x2_weights)
  int stage = 0, ahead = C::kStages - 1;
  for (int i = i0 + warp * C::kGroups; i < i1; i += W * C::kGroups) {
    st.fetch(ahead);
    if (++ahead == C::kStages) ahead = 0;
    cp_wait<C::kStages - 1>();
    __syncwarp();
    const unsigned held = st.fetched >> ((C::kStages - 1) * C::kGroups);  // group 0's bit highest
    const uint32_t base_at = ring + stage * C::kStage;
    // s[x]: elements 0, 1 are token g of heads 2t and 2t + 1, elements 2, 3 token g + 8
    float s[C::kGroups][NT][4];
#pragma unroll
    for (int x = 0; x < C::kGroups; ++x) {
      const uint32_t kt = base_at + x * 2 * C::kTile;
      if (!(held >> (C::kGroups - 1 - x) & 1u)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[x][n][0] = s[x][n][1] = s[x][n][2] = s[x][n][3] = -INFINITY;
        continue;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) s[x][n][0] = s[x][n][1] = s[x][n][2] = s[x][n][3] = 0.f;
      if constexpr (!FP8) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t r[4];
          ldsm4(kt + piece_at<C::kRowBytes>(lane & 15, 2 * ks + (lane >> 4)), r);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<false>(s[x][n], r, qf[n][ks][0], qf[n][ks][1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 w[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[h].x), "=r"(w[h].y), "=r"(w[h].z), "=r"(w[h].w)
                         : "r"(kt + piece_at<C::kRowBytes>(g + 8 * h, t + 4 * c))
                         : "memory");
          auto step = [&](int ks, uint32_t w0, uint32_t w1) {
            uint32_t r[4];
            e4m3x4_f16(w0, r[0], r[2]);
            e4m3x4_f16(w1, r[1], r[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16<true>(s[x][n], r, qf[n][4 * c + ks][0], qf[n][4 * c + ks][1]);
          };
          step(0, w[0].x, w[1].x);
          step(1, w[0].y, w[1].y);
          step(2, w[0].z, w[1].z);
          step(3, w[0].w, w[1].w);
        }
      }
      const int j0 = gr.at(i + x) * kPageStep;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][n][y] *= qs[n][y & 1];
      if (!gr.whole(j0)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (!sees(gr.seen, j0 + g + 8 * (y >> 1))) s[x][n][y] = -INFINITY;
      }
    }
    float top[NT][2];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = max_nan(s[0][n][h], s[0][n][2 + h]);
#pragma unroll
        for (int x = 1; x < C::kGroups; ++x) v = max_nan(v, max_nan(s[x][n][h], s[x][n][2 + h]));
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, k));
        top[n][h] = v;
        grew |= !(v <= m[n][h]);
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float now = max_nan(m[n][h], top[n][h]), f = m[n][h] == -INFINITY ? 0.f : exp2_approx(m[n][h] - now);
          m[n][h] = now;
          l[n][h] *= f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) o[n][c][h] *= f, o[n][c][2 + h] *= f;
        }
    }
#pragma unroll
    for (int x = 0; x < C::kGroups; ++x) {
      if (!(held >> (C::kGroups - 1 - x) & 1u)) continue;
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float b0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - kUp, b1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - kUp;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float e0 = exp2_approx(s[x][n][2 * h] - b0), e1 = exp2_approx(s[x][n][2 * h + 1] - b1);
          l[n][0] += e0;
          l[n][1] += e1;
          pf[n][h] = movm_t(FP8 ? f16x2_weights(e0, e1) : bf16x2_rn(e0, e1));
        }
      }
      const uint32_t vt = base_at + x * 2 * C::kTile + C::kTile;
      if constexpr (!FP8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t r[4];
          ldsm4_t(vt + piece_at<C::kRowBytes>((lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1)), r);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<false>(o[n][c], r, pf[n][0], pf[n][1]);
        }
      } else {
        // a register of the transposed load holds two columns of two tokens: sorted by
        // column they are rows g and g + 8 of the operand
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[4];
          ldsm4_t(vt + piece_at<C::kRowBytes>(lane & 15, 2 * c + (lane >> 4)), r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[4];
            e4m3x4_f16(__byte_perm(r[2 * h], 0, 0x3120), v[0], v[1]);
            e4m3x4_f16(__byte_perm(r[2 * h + 1], 0, 0x3120), v[2], v[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16<true>(o[n][2 * c + h], v, pf[n][0], pf[n][1]);
          }
        }
      }
    }
    __syncwarp();  // the stage is free for the next fetch
    if (++stage == C::kStages) stage = 0;
  }
  cp_wait<0>();

  // ---- the warps' sums joined, no longer scaled (v_scale / sum in that scale may leave fp32's range; taken out
  // at the output, 64 sequences of up to 16000 took 2 us more)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], k);
      if (g == 0) ml[warp][8 * n + 2 * t + h] = make_float2(m[n][h], l[n][h] * kDown);
    }
  __syncthreads();  // (every warp is done with the ring too)
  float* join = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * n + 2 * t + h;
      if (row < nq) {
        float* dst = join + (warp * C::kHeads + row) * C::kJoinLd;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          if constexpr (FP8) {
            *reinterpret_cast<float2*>(dst + 16 * c + 2 * g) = make_float2(o[n][c][h] * kDown, o[n][c][2 + h] * kDown);
          } else {
            dst[16 * c + g] = o[n][c][h];
            dst[16 * c + 8 + g] = o[n][c][2 + h];
          }
        }
      }
    }
  __syncthreads();
  constexpr int kHeads = 128 / D;
  for (int r0 = warp * kHeads; r0 < nq; r0 += W * kHeads) {
    const int row = r0 + (4 * lane) / D, col = (4 * lane) % D;
    Joined j = {make_float4(0, 0, 0, 0), -INFINITY, 0.f};
    if (row < nq) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        j.add(*reinterpret_cast<const float4*>(join + (w * C::kHeads + row) * C::kJoinLd + col), ml[w][row]);
    }
    done(r0, row, col, j);
  }
}

// Zeros for the sequences that see nothing.
__device__ __forceinline__ void zero_rows(const PagedAttn& a, int warp, int lane) {
  for (int b = blockIdx.x; b < a.batch.seqs; b += gridDim.x)
    if (groups_of(a, b).n == 0) {
      for (int col = 128 * warp; col < a.out.cols; col += 128 * kWarps)
        store_cols128(a.out, b, col, a.out.cols - col, lane, make_float4(0, 0, 0, 0));
    }
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kWarps, (DecCfg<D, FP8, NT, false>::kCtas)) decode_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[kWarps];
  __shared__ int64_t found_base;
  __shared__ int found_b;
  __shared__ float2 ml[kWarps][kRows];
  const PagedAttn& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's run of the units (sequence, head group, group of 16 tokens)
  const int B = a.batch.seqs, heads = a.kv.heads * p.hgroups, per = (B + 32 * kWarps - 1) / (32 * kWarps);
  const int b_first = min(B, tid * per), b_last = min(B, b_first + per);
  int64_t mine = 0;
  for (int b = b_first; b < b_last; ++b) mine += (int64_t)groups_of(a, b).n * heads;
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) scan[warp] = before;
  if (tid == 0) found_b = -1;
  __syncthreads();
  int64_t units = 0;
  before -= mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    units += scan[w];
  }
  const int64_t run = max((units + gridDim.x - 1) / gridDim.x, (int64_t)kMinRun);
  const int64_t u0 = min(units, blockIdx.x * run), u1 = min(units, u0 + run);
  if (before <= u0 && u0 < before + mine) {
    int64_t at = before;
    int b = b_first;
    for (;; ++b) {
      const int64_t n = (int64_t)groups_of(a, b).n * heads;
      if (u0 < at + n) break;
      at += n;
    }
    found_b = b;
    found_base = at;
  }
  if (tid == 0 && !p.by_segment) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  zero_rows(a, warp, lane);
  if (p.by_segment)
    for (int b = blockIdx.x; b < B; b += gridDim.x)
      if (groups_of(a, b).n == 0)
        for (int h = tid; h < heads; h += 32 * kWarps) p.joins[b * heads + h] = make_int4(0, 0, 0, 0);
  if (u0 >= u1) return;

  int b = found_b;
  Groups gr = groups_of(a, b);
  int hg = (int)((u0 - found_base) / gr.n);
  int64_t seg = found_base + (int64_t)hg * gr.n;  // first unit of this head
  for (int64_t u = u0; u < u1;) {
    const int64_t seg_end = seg + gr.n;
    const int i0 = (int)(u - seg), i1 = (int)(min(u1, seg_end) - seg);
    const int kh = hg / p.hgroups, sub = hg - kh * p.hgroups;
    const int qh = kh * a.group + sub * kRows, nq = min(kRows, a.group - sub * kRows);
    const bool begins = i0 == 0, ends = i1 == gr.n;
    const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
    attend<D, FP8, NT, false, kWarps>(a, gr, b, kh, qh, nq, i0, i1, smem, ml, [&](int r0, int row, int col, const Joined& j) {
      if (begins && ends) {
        store_cols128(a.out, b, (qh + r0) * D, (nq - r0) * D, lane, j.out(FP8 ? a.kv.v_scale[kh] : 1.f));
      } else if (row < nq) {
        *reinterpret_cast<float4*>(p.part + ((int64_t)slot * kRows + row) * D + col) = j.v;
        if (col == 0) p.ml[slot * kRows + row] = make_float2(j.top, j.sum);
      }
    });
    if (begins && tid == 0 && (p.by_segment || !ends))
      p.joins[p.by_segment ? b * heads + hg : (int)blockIdx.x] =
          make_int4(b, hg, ends ? 0 : (int)((seg_end - 1) / run) - (int)blockIdx.x + 1, (int)blockIdx.x);
    __syncthreads();  // the join region is the ring's again

    u = min(u1, seg_end);
    seg = seg_end;
    if (u < u1 && ++hg == heads) {
      hg = 0;
      do gr = groups_of(a, ++b);
      while (gr.n == 0);
    }
  }
}

// Short caches: a cluster of CTAs (or one) a sequence's head, joined through
// distributed shared memory.  One launch without a plan or a workspace: 700 tokens, 8
// heads 5.5 us, the other form 10.
template <int D, bool FP8, int NT, int W>
__global__ void __launch_bounds__(32 * W, (DecCfg<D, FP8, NT, true, W>::kCtas)) decode_cluster_kernel(const __grid_constant__ DecodeParams p) {
  using C = DecCfg<D, FP8, NT, true, W>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 ml[W][kRows], all_ml[kRows];
  const PagedAttn& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), S = p.cluster, seg = blockIdx.x / S;
  pdl_wait();
  pdl_trigger();
  const int heads = a.kv.heads * p.hgroups, b = seg / heads, hg = seg - b * heads;
  const int kh = hg / p.hgroups, sub = hg - kh * p.hgroups;
  const int qh = kh * a.group + sub * kRows, nq = min(kRows, a.group - sub * kRows);
  const Groups gr = groups_of(a, b);
  // (parts of whole steps of all warps, so that a short cache is not spread too thin)
  constexpr int kStep = W * C::kGroups;
  const int steps = (gr.n + kStep - 1) / kStep;
  const int i0 = min(gr.n, steps * rank / S * kStep), i1 = min(gr.n, steps * (rank + 1) / S * kStep);
  float* part = reinterpret_cast<float*>(smem + C::kJoin);
  const float v_scale = FP8 ? a.kv.v_scale[kh] : 1.f;
  attend<D, FP8, NT, true, W>(a, gr, b, kh, qh, nq, i0, i1, smem, ml, [&](int r0, int row, int col, const Joined& j) {
    if (S == 1) {
      store_cols128(a.out, b, (qh + r0) * D, (nq - r0) * D, lane, j.out(v_scale));
    } else if (row < nq) {
      *reinterpret_cast<float4*>(part + row * D + col) = j.v;
      if (col == 0) all_ml[row] = make_float2(j.top, j.sum);
    }
  });
  if (S == 1) return;
  cluster_arrive_wait();
  constexpr int kHeads = 128 / D;
  for (int r0 = (rank * W + warp) * kHeads; r0 < nq; r0 += S * W * kHeads) {
    const int row = r0 + (4 * lane) / D, col = (4 * lane) % D;
    Joined j = {make_float4(0, 0, 0, 0), -INFINITY, 0.f};
    if (row < nq) {
      float4 x[kMaxCluster];
      float2 m[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        m[r] = make_float2(-INFINITY, 0.f);
        x[r] = make_float4(0, 0, 0, 0);
        if (r < S) {
          asm volatile(
              "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %4, %5;\n\t"
              "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
              : "=f"(x[r].x), "=f"(x[r].y), "=f"(x[r].z), "=f"(x[r].w)
              : "r"(smem_u32(part + row * D + col)), "r"(r)
              : "memory");
          asm volatile(
              "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %2, %3;\n\t"
              "ld.shared::cluster.v2.f32 {%0, %1}, [ra];\n\t}"
              : "=f"(m[r].x), "=f"(m[r].y)
              : "r"(smem_u32(&all_ml[row])), "r"(r)
              : "memory");
        }
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) j.add(x[r], m[r]);
    }
    store_cols128(a.out, b, (qh + r0) * D, (nq - r0) * D, lane, j.out(v_scale));
  }
  cluster_arrive_wait();  // the others may still read this CTA's part
}

// Joins the runs of one head that lies in several: block (entry of joins,
// 128 columns of its rows); each warp adds every fourth run's sums, four columns a
// lane.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kHeads = 128 / D, kW = 4, kAhead = 8;
  __shared__ float4 sums[kW][32];
  __shared__ float2 mls[kW][kHeads];
  pdl_wait();
  pdl_trigger();
  const int4 d = p.joins[blockIdx.x];
  if (d.z == 0) return;
  const PagedAttn& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = d.y / p.hgroups, sub = d.y - kh * p.hgroups;
  const int qh = kh * a.group + sub * kRows, nq = min(kRows, a.group - sub * kRows);
  const int r0 = blockIdx.y * kHeads;
  if (r0 >= nq) return;
  const int head = (4 * lane) / D, row = r0 + head, col = (4 * lane) % D;
  Joined j = {make_float4(0, 0, 0, 0), -INFINITY, 0.f};
  if (row < nq)
    for (int i0 = warp; i0 < d.z; i0 += kAhead * kW) {
      float2 ml[kAhead];
      float4 x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + kW * k;
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0, 0, 0, 0);
        if (i < d.z) {
          const int slot = 2 * (d.w + i) + (i == 0);
          ml[k] = p.ml[slot * kRows + row];
          x[k] = *reinterpret_cast<const float4*>(p.part + ((int64_t)slot * kRows + row) * D + col);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) j.add(x[k], ml[k]);
    }
  sums[warp][lane] = j.v;
  if (col == 0) mls[warp][head] = make_float2(j.top, j.sum);
  __syncthreads();
  if (warp) return;
  j = {make_float4(0, 0, 0, 0), -INFINITY, 0.f};
#pragma unroll
  for (int w = 0; w < kW; ++w) j.add(sums[w][lane], mls[w][head]);
  store_cols128(a.out, d.x, (qh + r0) * D, (nq - r0) * D, lane, j.out(FP8 ? a.kv.v_scale[kh] : 1.f));
}

constexpr int kSms = 152, kMaxGrid = 4 * kSms;  // CTAs: up to four an SM

// Sequences' heads (and groups of 16 query heads).
int64_t segments_of(const PagedAttn& a) { return (int64_t)a.batch.seqs * a.kv.heads * ((a.group + kRows - 1) / kRows); }

// Cached tokens of a sequence that are read, at most: whole groups of 16 of the window and the sinks.
int64_t tokens_of(const PagedAttn& a) {
  const int64_t step = kPageStep, seen = ((a.window + step - 1) / step + 1 + (a.sinks + step - 1) / step) * step;
  return a.window > 0 ? std::min((int64_t)a.batch.reach, seen) : a.batch.reach;
}

// CTAs of decode_cluster_kernel that an SM holds.
constexpr int cluster_ctas(int head_dim, int group) { return group > 8 ? 2 : head_dim == 128 ? 3 : 4; }

// CTAs of decode_cluster_kernel a sequence's head; 0: decode_kernel.  The one takes no
// plan, no workspace and no second launch, and CTAs take up heads as others end; as many
// a head as all run at once (24 sequences of up to 1900, 8 heads: two 22 us, one 28).  But a
// long sequence among short ones keeps its CTAs long after the others have ended, and E4M3
// streams run faster in the other form, so each may have 2048 tokens of a head of 128 at most (64
// sequences of 3900, 8 heads, E4M3: 85 us, as clusters of one 107; 48 of up to 1900, bf16: 43 us, as
// clusters 37), twice that of 64 (64 of 4095, 8 heads: 89 us, as clusters 84).
int cluster_of(const PagedAttn& a, int head_dim) {
  const int64_t segments = segments_of(a);
  const int64_t tokens = tokens_of(a), steps = (tokens + 16 * kWarps - 1) / (16 * kWarps);  // steps: of all warps, 16 tokens each
  int n = 1;
  while (n < kMaxCluster && segments * 2 * n <= cluster_ctas(head_dim, a.group) * kSms && n < steps) n *= 2;
  return tokens * head_dim <= (int64_t)n * kClusterValues ? n : 0;
}

template <int D, bool FP8, int NT, int W>
cudaError_t launch_cluster(const DecodeParams& p, cudaStream_t s) {
  using C = DecCfg<D, FP8, NT, true, W>;
  static_assert(C::kCtas * W == cluster_ctas(D, 8 * NT) * kWarps);
  static bool attr_set[64] = {};
  if (cudaError_t e = allow_smem(decode_cluster_kernel<D, FP8, NT, W>, C::kSmem, attr_set)) return e;
  return launch_pdl_cluster(decode_cluster_kernel<D, FP8, NT, W>, dim3((unsigned)(segments_of(p.a) * p.cluster)), dim3(32 * W),
                            C::kSmem, s, (unsigned)p.cluster, p);
}

template <int D, bool FP8, int NT>
cudaError_t launch(const PagedAttn& a, void* ws, cudaStream_t s) {
  DecodeParams p;
  p.a = a;
  p.hgroups = (a.group + kRows - 1) / kRows;
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.part = reinterpret_cast<float*>(at);
  at += (size_t)kMaxGrid * 2 * kRows * D * 4;
  p.ml = reinterpret_cast<float2*>(at);
  at += (size_t)kMaxGrid * 2 * kRows * 8;
  p.joins = reinterpret_cast<int4*>(at);
  p.cluster = cluster_of(a, D);
  // Many heads of short caches: CTAs of two warps, twice as many at once (256 sequences of 30, 8 heads:
  // 17 -> 12 us, 64 of 500 28 -> 24; but 128 of up to 1000 47 -> 50).
  if (p.cluster)
    return p.cluster == 1 && tokens_of(a) <= 512 ? launch_cluster<D, FP8, NT, 2>(p, s) : launch_cluster<D, FP8, NT, kWarps>(p, s);
  using C = DecCfg<D, FP8, NT, false>;
  constexpr int kGrid = C::kCtas * kSms;
  static bool attr_set[64] = {};
  if (cudaError_t e = allow_smem(decode_kernel<D, FP8, NT>, C::kSmem, attr_set)) return e;
  p.by_segment = segments_of(a) <= kGrid;  // (fewer blocks: most of the join's would find nothing)
  if (cudaError_t e = launch_pdl(decode_kernel<D, FP8, NT>, dim3(kGrid), dim3(32 * kWarps), C::kSmem, s, p)) return e;
  const unsigned blocks = (unsigned)((std::min(a.group, kRows) * D + 127) / 128);
  return launch_pdl(decode_join_kernel<D, FP8>, dim3((unsigned)(p.by_segment ? segments_of(a) : kGrid), blocks), dim3(128), 0, s, p);
}

template <int D, bool FP8>
cudaError_t launch_heads(const PagedAttn& a, void* ws, cudaStream_t s) {
  return a.group <= 8 ? launch<D, FP8, 1>(a, ws, s) : launch<D, FP8, 2>(a, ws, s);
}

}  // namespace

bool attn_decode_needs_workspace(const PagedAttn& a, int head_dim) { return cluster_of(a, head_dim) == 0; }

size_t attn_decode_workspace(int head_dim) { return (size_t)kMaxGrid * (2 * kRows * (head_dim * 4 + 8) + 16); }

cudaError_t launch_attn_decode(const PagedAttn& a, int head_dim, bool fp8, void* ws, cudaStream_t s) {
  if (head_dim == 64) return fp8 ? launch_heads<64, true>(a, ws, s) : launch_heads<64, false>(a, ws, s);
  return fp8 ? launch_heads<128, true>(a, ws, s) : launch_heads<128, false>(a, ws, s);
}

}  // namespace fp4moe
