// Block-scaled FP8 linear for many tokens on the tensor cores (tcgen05,
// E4M3 x E4M3, fp32 accumulators in tensor memory).
//
// The scales change every 128 columns of K and are arbitrary fp32 numbers, so
// they cannot ride in the MMA: each K block's product goes to a buffer of tensor
// memory (two of 256 columns, four of 128), and the epilogue warps fold it,
// times xs[t, b] ws[n / 128, b], into fp32 sums held in their registers while the
// MMAs of the next blocks fill the other buffers.  Lanes are tokens, so a
// thread's factor is one number a block: one fused multiply-add per element, two
// to an instruction.
//
// What bounds it: shared memory.  A K block of a 128 x 256 tile writes 48 KB of
// operands there and the MMAs read them again, 768 cycles at 128 bytes a cycle
// against 512 of the tensor core (fp8); measured 780 without the epilogue's
// sums, 840 with them (16384 x 7168 x 7168 in 583 us, 2.89 PFLOP/s).  Run for
// seconds the board's power cap takes the clock to 1.6 GHz: 670 us.  CTA pairs
// (256 x 256 over two SMs, 512 cycles of shared memory) reached 474 us without
// the sums but 615 with them: two buffers of tensor memory are then too few for
// the way round over both CTAs.  Operands multicast to two CTAs changed nothing.
//
// Work split: with about a tile or more for every SM, persistent CTAs take whole
// tiles in turn, 256 weight rows wide where that fills whole rounds and 128
// wide for the rest (a launch of its own that starts where the first one's
// CTAs run out of tiles).  With fewer, a cluster of S CTAs shares a tile, each
// with a run of its K blocks; each sends the others their slices of the columns
// through distributed shared memory and adds its own over the runs, in the order
// of K.
//
// Warp roles: warp 0 TMA producer, warps 1 and 2 MMA issuers, warps 4-11 epilogue
// (warp groups of their own, with the larger register share).  Every wait on a
// barrier in shared memory is bounded; a timeout records FP4MOE_ERR_TIMEOUT in the
// status word, drains copies and MMAs in flight, frees tensor memory and returns.
// The two cluster barriers of a shared tile have no limit of their own: a CTA
// comes to both whether its roles finished or gave up, so their peers wait as
// long as the bounded waits may.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "fp8_block.cuh"
#include "internal.h"

namespace fp4moe {

namespace {

// Where calls without a workspace record a timeout; cleared when it is read.
__device__ int32_t linear_status[kStatusInts];

// Tiles of one launch: 128 tokens x BN rows of W.
struct TcPlan {
  int split;              // CTAs that share a tile
  int nb;                 // K blocks
  int mtiles, ntiles;
};
constexpr int kTcCtas = 152;    // one CTA per SM

struct TcParams {
  CUtensorMap tmx, tmw;    // boxes of whole tiles
  CUtensorMap tmx1, tmw1;  // the last token tile's and the last weight tile's: the rows that exist
  const float *xs, *ws;
  uint8_t* out;
  int64_t out_ld;
  int32_t* status;        // null: linear_status
  TcPlan plan;
  int T, N;
  int xbytes, wbytes;     // of the last tiles' boxes
  int out_fp32, vec;      // vec: 16-byte stores are aligned
  int second;             // the second launch of a call: joins the first one's end, not its start
  int withhold;           // test knob: CTA 0 never fills its first stage
  uint64_t wait_ns;       // limit of the pipeline's waits (drains keep kWaitLimitNs)
};

template <int BN, bool SPLIT>
struct TcCfg {
  static constexpr int kEpiWarps = 8, kThreads = 128 + 32 * kEpiWarps;  // warp 3 idles
  static constexpr int kCols = BN / 2;  // columns of one epilogue warp
  static constexpr int kABytes = 128 * 128, kBBytes = BN * 128, kStage = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 4 : SPLIT ? 5 : 6;
  static constexpr int kBufs = 512 / BN;              // all of tensor memory
  // 32 rows x 128 bytes per epilogue warp; SPLIT: the other CTAs' sums of this one's slice, 7/8 of a tile at most
  static constexpr int kStaging = SPLIT ? 128 * BN * 4 * 7 / 8 : kEpiWarps * 4096;
  static constexpr int kSmem = kStages * kStage + kStaging + 1024;
  // launched with 168 registers a thread (384 threads); 128 x 40 + 256 x 232 = 384 x 168
  static constexpr int kCtlRegs = 40, kEpiRegs = 232;
};

__device__ __forceinline__ uint64_t desc_sw128_k(uint32_t saddr) { return smem_desc(saddr, 16, 1024, 2); }

// 16 tensor-memory columns of this thread's lane, in flight until tmem_landed16.
__device__ __forceinline__ void tmem_fetch16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Waits for every fetch of this thread; naming the registers keeps their uses behind the wait.
__device__ __forceinline__ void tmem_landed16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
// acc += a * s, two fp32 lanes in one instruction.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(s));
}

// The box of a 2-D tensor map at (x, y) on its way into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* m, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(m), "r"(x), "r"(y) : "memory");
}

// The two halves of cluster_arrive_wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 16 bytes to this CTA's shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t addr, int rank, const uint32_t* v) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
      "st.shared::cluster.v4.b32 [ra], {%2, %3, %4, %5};\n\t}" ::"r"(addr),
      "r"(rank), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
      : "memory");
}

// A scale load that stays where it is written (volatile): moved down to its
// first use, its whole latency would show in every K block.  A plain load: the
// read-only path asks for memory that nothing writes while this kernel runs, and
// the launch before, which may write the scales, ends after this one has begun.
__device__ __forceinline__ float fetch1(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// Tile order: groups of kGroupM token tiles, each group over every weight
// tile, so that the tiles running at one time share both operands in L2.
constexpr int kGroupM = 8;
__device__ __forceinline__ void tile_at(int tile, int mtiles, int ntiles, int& mt, int& nt) {
  const int per = kGroupM * ntiles, g = tile / per, in = tile - g * per;
  const int gm = min(kGroupM, mtiles - g * kGroupM);
  nt = in / gm;
  mt = g * kGroupM + in - nt * gm;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void store_one(const TcParams& p, uint8_t* d, uint32_t v) {
  if (p.out_fp32)
    *reinterpret_cast<uint32_t*>(d) = v;
  else
    *reinterpret_cast<uint16_t*>(d) = (uint16_t)v;
}

// The 16 bytes of (lo, hi) from byte `at`, an even number below 16.
__device__ __forceinline__ uint4 bytes_from(const uint4& lo, const uint4& hi, int at) {
  uint32_t w[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  if (at & 8) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = w[6], w[5] = hi.w;
  if (at & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
  const uint32_t sh = (at & 2) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                    __funnelshift_r(w[3], w[4], sh));
}

// One warp's 32 staged rows (at shared-memory address stg, 128 bytes each, 16-byte
// pieces xor-swizzled by the row) to columns [col, col + cols) of rows row.. of
// out, where these are inside it.  Eight lanes a row, whole aligned 16-byte
// vectors; a row of an odd width starts anywhere, so its vectors are put together
// from two pieces, and what sticks out of them at either end goes element by
// element (eight of bf16 in 128 bytes: one a lane).  Loads of several rows
// before their stores: one row at a time waits for shared memory each time.
__device__ __forceinline__ void store_rows(const TcParams& p, uint32_t stg, int lane, int row, int col, int cols) {
  const int esz = p.out_fp32 ? 4 : 2, nbytes = min(cols, p.N - col) * esz, nrow = min(32, p.T - row);
  if (nbytes <= 0) return;
  uint8_t* dst = p.out + ((int64_t)row * p.out_ld + col) * esz;
  const int64_t ld = p.out_ld * esz;
  const int l = lane & 7, r0 = lane >> 3;
  if (p.vec && nbytes % 16 == 0) {
    uint8_t* d = dst + r0 * ld + 16 * l;
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = lds128(stg + (r0 + 4 * i) * 128 + ((l ^ ((r0 + 4 * i) & 7)) << 4));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + 4 * i < nrow && 16 * l < nbytes) *reinterpret_cast<uint4*>(d + 4 * i * ld) = w[i];
    return;
  }
  // Of a row that starts off bytes into a vector, the window's first n16 bytes are
  // n16 / 16 - 1 whole vectors, and of the elements of its first and last piece
  // those outside them: 16 bytes together.
  const int n16 = nbytes & ~15, rest = n16 + l * esz;
  uint8_t* d = dst + r0 * ld;
  const uint32_t row_at = stg + r0 * 128;
  constexpr int kRows = 4;  // a lane's rows at a time
#pragma unroll
  for (int h = 0; h < 8; h += kRows) {
    uint4 lo[kRows], hi[kRows];
    uint32_t e[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t at = row_at + 512 * (h + i), x = (r0 + 4 * i) & 7;  // (its swizzle)
      const int off = (int)(reinterpret_cast<uintptr_t>(d + 4 * i * ld) & 15u), eb = l * esz;
      lo[i] = lds128(at + ((l ^ x) << 4));
      hi[i] = lds128(at + (((l + 1) & 7) ^ x) * 16);
      const int piece = eb < 16 - off ? 0 : (n16 >> 4) - 1;
      e[i] = lds32(at + (((piece & 7) ^ x) << 4) + (eb & 12)) >> ((eb & 2) * 8);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + 4 * (h + i), eb = l * esz;
      const int off = (int)(reinterpret_cast<uintptr_t>(d) & 15u), head = (16 - off) & 15;
      if (r < nrow) {
        if (16 * l < n16 - (off ? 16 : 0)) *reinterpret_cast<uint4*>(d + head + 16 * l) = bytes_from(lo[i], hi[i], head);
        if (off && eb < 16 && n16) store_one(p, d + (eb < head ? eb : n16 - 16 + eb), e[i]);
        if (rest < nbytes)
          store_one(p, d + rest,
                    lds32(row_at + 512 * (h + i) + (((rest >> 4) ^ r) & 7) * 16 + (rest & 12)) >> ((rest & 2) * 8));
      }
      d += 4 * ld;
    }
  }
}

// A cluster's join.  Of a tile's COLS columns of this thread's row (acc: pairs) a
// slice falls to each of the S CTAs: a thread sends the others theirs, then sums
// its own over the CTAs in the order of K.  `at`: vector 0 of this thread in
// the region for the others' sums, where CTA s of the others has the s-th part.
// Sent, not fetched: with the loads of a slice from every CTA the join took 4.5
// us, with stores 2.2 (128 x 7168 x 7168, two CTAs a tile: 17.5 -> 16.1 us; 333 x 7168 x
// 2000, four: 15.7 -> 13.1).
template <int COLS, int S>
__device__ __forceinline__ void join_slices(const TcParams& p, const uint64_t* acc, uint32_t at, uint8_t* stg, int rank,
                                            int lane, int row, int col) {
  constexpr int kVecs = COLS / 4 / S;  // of 4 columns
  uint32_t own[kVecs][4];
#pragma unroll
  for (int r = 0; r < S; ++r)
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint32_t w[4];
      unpack2(acc[2 * (kVecs * r + i)], w[0], w[1]);
      unpack2(acc[2 * (kVecs * r + i) + 1], w[2], w[3]);
      if (r == rank) {
#pragma unroll
        for (int j = 0; j < 4; ++j) own[i][j] = w[j];
      } else if (row + lane < p.T) {
        st_cluster(at + 4096u * (kVecs * (rank - (rank > r)) + i), r, w);
      }
    }
  __syncwarp();
  cluster_arrive_wait();
  float v[4 * kVecs];
#pragma unroll
  for (int j = 0; j < 4 * kVecs; ++j) v[j] = 0.f;
#pragma unroll
  for (int r = 0; r < S; ++r)
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint32_t w[4];
      if (r == rank) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = own[i][j];
      } else {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at + 4096u * (kVecs * (r - (r > rank)) + i))
                     : "memory");
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] += __uint_as_float(w[j]);
    }
  // 4 kVecs columns of 32 rows, through shared memory
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (p.out_fp32)
      *reinterpret_cast<float4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else if (i % 2 == 0)
      *reinterpret_cast<uint4*>(stg + lane * 128 + (((i / 2) ^ (lane & 7)) << 4)) =
          make_uint4(bf16x2_rn(v[4 * i], v[4 * i + 1]), bf16x2_rn(v[4 * i + 2], v[4 * i + 3]),
                     bf16x2_rn(v[4 * i + 4], v[4 * i + 5]), bf16x2_rn(v[4 * i + 6], v[4 * i + 7]));
  }
  __syncwarp();
  store_rows(p, smem_u32(stg), lane, row, col + 4 * kVecs * rank, 4 * kVecs);
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(TcCfg<BN, SPLIT>::kThreads, 1) linear_tc_kernel(const __grid_constant__ TcParams p) {
  using C = TcCfg<BN, SPLIT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages];
  __shared__ __align__(8) uint64_t bar_tfull[C::kBufs], bar_tempty[C::kBufs], bar_done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // SPLIT: one tile a cluster, K blocks [kb0, kb1) in this CTA; else tiles
  // blockIdx.x, + gridDim.x, ... whole
  const int S = SPLIT ? p.plan.split : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / S, step = (int)gridDim.x / S, tiles = p.plan.mtiles * p.plan.ntiles;
  const int kb0 = SPLIT ? p.plan.nb * rank / S : 0, kb1 = SPLIT ? p.plan.nb * (rank + 1) / S : p.plan.nb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    for (int a = 0; a < C::kBufs; ++a) {
      mbar_init(smem_u32(&bar_tfull[a]), 1);
      mbar_init(smem_u32(&bar_tempty[a]), C::kEpiWarps);
    }
    mbar_init(smem_u32(&bar_done), 2);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.tmx);
    prefetch_tmap(&p.tmw);
    prefetch_tmap(&p.tmx1);
    prefetch_tmap(&p.tmw1);
    // One token tile: the first weight boxes on their way into L2 while the launch
    // before ends (16 x 7168 x 36864 43.6 -> 42.1 us; with more token tiles no gain).
    if (p.plan.mtiles == 1 && first < tiles) {
      const CUtensorMap* tmw = first + 1 == tiles ? &p.tmw1 : &p.tmw;
      for (int kb = kb0; kb < min(kb1, kb0 + 3); ++kb) tma_prefetch_2d(tmw, kb * 128, first * BN);
    }
  }
  // The second launch of a call begins once every CTA of the first has passed
  // its own wait, so its inputs are complete; it waits for the first at its end,
  // so that whoever waits for the second waits for both.
  if (!p.second) {
    pdl_wait();
    if (p.status && blockIdx.x == 0 && threadIdx.x < kStatusInts) p.status[threadIdx.x] = 0;
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if constexpr (SPLIT) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort_v = &abort_flag;
  auto timed_out = [&]() {  // by one lane
    if (!*abort_v) record_status(p.status ? p.status : linear_status, FP4MOE_ERR_TIMEOUT, ST_TIMEOUT);
    *abort_v = 1;
  };
  // bounded wait with a warp-uniform outcome
  auto wait_w = [&](uint32_t bar, uint32_t par) {
    return __all_sync(0xffffffffu, mbar_wait_abortable(bar, par, p.wait_ns, abort_v)) != 0;
  };

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kCtlRegs));
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = p.withhold && blockIdx.x == 0 ? 1 : 0, kb = kb0 + stage;
      uint32_t phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int tile = first; ok && tile < tiles; tile += step) {
        int mt, nt;
        tile_at(tile, p.plan.mtiles, p.plan.ntiles, mt, nt);
        // Boxes end with the rows that exist.  What shared memory holds past them goes
        // through the MMAs into rows and columns that are not stored.  (Boxes of whole
        // tiles, zeros filled in past the end, arrive at half the rate: 16 x 7168 x
        // 18432 took 33 us, now 24.)
        const bool x1 = mt + 1 == p.plan.mtiles, w1 = nt + 1 == p.plan.ntiles;
        const CUtensorMap *tmx = x1 ? &p.tmx1 : &p.tmx, *tmw = w1 ? &p.tmw1 : &p.tmw;
        const uint32_t bytes = (x1 ? p.xbytes : C::kABytes) + (w1 ? p.wbytes : C::kBBytes);
        for (; kb < kb1; ++kb) {
          if (!mbar_wait_abortable(smem_u32(&bar_empty[stage]), phase ^ 1u, p.wait_ns, abort_v)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&bar_full[stage]), base = sbase + stage * C::kStage;
          mbar_arrive_expect_tx(fb, bytes);
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          tma_load_2d(base, tmx, fb, kb * 128, mt * 128);
          tma_load_2d(base + C::kABytes, tmw, fb, kb * 128, nt * BN);
          if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        }
        kb = kb0;
      }
      if (!ok) timed_out();
      for (int s = 0; s < C::kStages; ++s)  // every armed stage lands before the CTA exits
        if ((armed >> s) & 1u) (void)mbar_wait(smem_u32(&bar_full[s]), (armed_par >> s) & 1u);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers
    // Two, for the even and the odd K blocks: issuing a block's four MMAs and its
    // two commits takes one warp longer than the tensor core needs for it (128-wide
    // tiles 968 -> 801 us at 16384 x 7168 x 7168).
    const uint64_t a0 = desc_sw128_k(sbase), b0 = desc_sw128_k(sbase + C::kABytes);
    int stage = warp - 1, buf = warp - 1;
    uint32_t phase = 0, bphase = 0;
    bool ok = true;
    int mine = warp - 1;  // K blocks to pass by before this warp's next one
    for (int tile = first; ok && tile < tiles; tile += step) {
      int kb = kb0 + mine;
      for (; kb < kb1; kb += 2) {
        if (!wait_w(smem_u32(&bar_tempty[buf]), bphase ^ 1u) || !wait_w(smem_u32(&bar_full[stage]), phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t so = (uint64_t)((stage * C::kStage) >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)  // K = 32 per MMA, 32 bytes of the 128-byte swizzle row
          tc_mma_f8_elect(tmem + buf * BN, a0 + so + 2 * j, b0 + so + 2 * j, idesc_f8(BN), j ? 1u : 0u);
        tc_commit_elect(smem_u32(&bar_empty[stage]));
        tc_commit_elect(smem_u32(&bar_tfull[buf]));
        stage += 2;
        if (stage >= C::kStages) { stage -= C::kStages; phase ^= 1u; }
        buf += 2;
        if (buf >= C::kBufs) { buf -= C::kBufs; bphase ^= 1u; }
      }
      mine = kb - kb1;
    }
    // all issued MMAs must finish before tensor memory is released
    tc_commit_elect(smem_u32(&bar_done));
    (void)mbar_wait(smem_u32(&bar_done), 0);
    if (!ok && lane == 0) timed_out();
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));
    const int q = warp & 3;                           // tensor-memory lane quadrant of this warp
    const int c0 = ((warp - 4) >> 2) * C::kCols;      // its columns
    uint8_t* stg = smem_raw + (sbase - smem_u32(smem_raw)) + C::kStages * C::kStage + (warp - 4) * 4096;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + c0;
    int buf = 0, t0 = 0, n0 = 0;
    uint32_t bphase = 0;
    bool ok = true;
    const float *xs = nullptr, *ws = nullptr;
    // the next K blocks' factors, fetched two blocks ahead (across tiles too)
    float fx[2], fw[2];
    auto open_tile = [&](int tile) {
      int mt, nt;
      tile_at(tile, p.plan.mtiles, p.plan.ntiles, mt, nt);
      t0 = mt * 128 + 32 * q;
      n0 = nt * BN + c0;
      xs = p.xs + (int64_t)min(t0 + lane, p.T - 1) * p.plan.nb;
      ws = p.ws + (int64_t)(min(n0, p.N - 1) / kBlk) * p.plan.nb;
#pragma unroll
      for (int i = 0; i < 2; ++i) fx[i] = fetch1(xs + min(kb0 + i, kb1 - 1)), fw[i] = fetch1(ws + min(kb0 + i, kb1 - 1));
    };
    uint64_t acc[C::kCols / 2];  // pairs of columns
    if (first < tiles) open_tile(first);
    for (int tile = first; tile < tiles; tile += step) {
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const float f = fx[0] * fw[0];
        const uint64_t f2 = pack2(__float_as_uint(f), __float_as_uint(f));
        fx[0] = fx[1], fw[0] = fw[1];
        if (kb + 2 < kb1) fx[1] = fetch1(xs + kb + 2), fw[1] = fetch1(ws + kb + 2);
        if (!wait_w(smem_u32(&bar_tfull[buf]), bphase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[2][16];
        tmem_fetch16(tq + buf * BN, v[0]);
#pragma unroll
        for (int c = 0; c < C::kCols / 16; ++c) {
          tmem_landed16(v[c & 1]);
          if (c + 1 < C::kCols / 16) {
            tmem_fetch16(tq + buf * BN + 16 * (c + 1), v[(c + 1) & 1]);
          } else {  // the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_tempty[buf]));
            if (++buf == C::kBufs) { buf = 0; bphase ^= 1u; }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) fma2(acc[8 * c + j], pack2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), f2);
        }
      }
      if (!ok) break;
      if constexpr (SPLIT) break;
      const int st0 = t0, sn0 = n0;
      if (tile + step < tiles) open_tile(tile + step);
      // through shared memory (16-byte pieces xor-swizzled by the row), so
      // that a store covers whole 128-byte runs of a row
      const int per = p.out_fp32 ? 32 : 64;
#pragma unroll
      for (int o = 0; o < C::kCols / 32; ++o) {  // 32 fp32 columns at a time; bf16 takes 64
        if (!p.out_fp32 && o >= C::kCols / 64) break;
        const int nc = sn0 + o * per;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w[4];
          if (p.out_fp32) {
            unpack2(acc[16 * o + 2 * c], w[0], w[1]);
            unpack2(acc[16 * o + 2 * c + 1], w[2], w[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t lo, hi;
              unpack2(acc[(32 * o + 4 * c + i) % (C::kCols / 2)], lo, hi);
              w[i] = bf16x2_rn(__uint_as_float(lo), __uint_as_float(hi));
            }
          }
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        store_rows(p, smem_u32(stg), lane, st0, nc, per);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) timed_out();
    __syncwarp();
    if constexpr (SPLIT) {
      cluster_wait();  // every CTA of the cluster has begun
      const uint32_t at = sbase + C::kStages * C::kStage + 16u * (threadIdx.x - 128);
      stg = smem_raw + (sbase - smem_u32(smem_raw)) + (warp - 4) * 4096;  // the pipeline's stages have been read
      if (S == 2) join_slices<C::kCols, 2>(p, acc, at, stg, rank, lane, t0, n0);
      if (S == 4) join_slices<C::kCols, 4>(p, acc, at, stg, rank, lane, t0, n0);
      if (S == 8) join_slices<C::kCols, 8>(p, acc, at, stg, rank, lane, t0, n0);
    }
  }
  if constexpr (SPLIT) {
    if (warp < 4) {
      __syncwarp();
      cluster_wait();
      cluster_arrive_wait();
    }
  }

  // (SPLIT: the cluster's barrier, after every CTA's last fetch from tensor memory and last store to another)
  tc_fence_before();
  if constexpr (!SPLIT) __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (p.second) pdl_wait();
}

template <int BN, bool SPLIT>
cudaError_t launch_tc(const LinearFp8Args& a, int split, bool second, cudaStream_t s) {
  using C = TcCfg<BN, SPLIT>;
  auto k = linear_tc_kernel<BN, SPLIT>;
  TcParams p;
  memset(&p, 0, sizeof(p));
  p.plan = {split, blocks128(a.K), (a.T + 127) / 128, (a.N + BN - 1) / BN};
  const uint32_t xrows = (uint32_t)(a.T - 128 * (p.plan.mtiles - 1)), wrows = (uint32_t)(a.N - BN * (p.plan.ntiles - 1));
  p.xbytes = (int)(128 * xrows);
  p.wbytes = (int)(128 * wrows);
  auto map = [&](CUtensorMap* m, const uint8_t* base, int rows, uint32_t box_rows) {
    const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)rows}, strides[1] = {(uint64_t)a.K};
    const uint32_t box[2] = {128, box_rows};
    return encode_tmap_u8(m, base, 2, dims, strides, box, true);
  };
  if (!map(&p.tmx1, a.xq, a.T, xrows) || !map(&p.tmw1, a.w, a.N, wrows)) return cudaErrorInvalidValue;
  p.tmx = p.tmx1;
  p.tmw = p.tmw1;
  if (p.plan.mtiles > 1 && xrows != 128 && !map(&p.tmx, a.xq, a.T, 128)) return cudaErrorInvalidValue;
  if (p.plan.ntiles > 1 && wrows != BN && !map(&p.tmw, a.w, a.N, BN)) return cudaErrorInvalidValue;
  p.xs = a.xs;
  p.ws = a.ws;
  p.out = static_cast<uint8_t*>(a.out);
  p.out_ld = a.out_ld;
  p.status = static_cast<int32_t*>(a.scratch);
  p.T = a.T;
  p.N = a.N;
  p.out_fp32 = a.out_fp32 ? 1 : 0;
  p.vec = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && a.out_ld * (a.out_fp32 ? 4 : 2) % 16 == 0;
  p.second = second ? 1 : 0;
  p.withhold = a.withhold && !second;
  p.wait_ns = a.wait_ns ? a.wait_ns : kWaitLimitNs;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int64_t tiles = (int64_t)p.plan.mtiles * p.plan.ntiles;
  if constexpr (SPLIT)
    return launch_pdl_cluster(k, dim3((unsigned)(tiles * split)), dim3(C::kThreads), C::kSmem, s, (unsigned)split, p);
  // (the second launch: a CTA per tile, taken up as the first one's CTAs leave)
  return launch_pdl(k, dim3((unsigned)(second ? tiles : std::min<int64_t>(tiles, kTcCtas))), dim3(C::kThreads), C::kSmem, s,
                    p);
}

// How a call is run: columns [0, wide) in tiles of 256, the rest in tiles of
// 128; split > 1: all of it in tiles of 128 shared by `split` CTAs.  Chosen by
// the time per K block of a tile (measured: 0.43 us 256 wide, 0.29 us 128
// wide; joining a split tile 1.5 us for few tokens, 2.9 for 128) and the rounds
// that the tiles make on 152 SMs.  A split tile's CTAs are a cluster, and no more
// clusters are taken than run at the same time (measured: 15 of 8, 36 and more
// of 4, 76 of 2; with more, a second round doubles the time).
struct TcChoice {
  int wide, split;
  int64_t cost;  // in 10 ns, without the launch
};
TcChoice choose(int T, int K, int N) {
  constexpr int64_t kT256 = 43, kT128 = 29;  // 10 ns
  const int64_t join = 130 + std::min(T, 128) * 5 / 4;
  const int64_t nb = blocks128(K), mt = (T + 127) / 128, sms = kTcCtas;
  const int64_t n128 = (N + 127) / 128;
  TcChoice best{0, 1, 0};
  int64_t cost = (mt * n128 + sms - 1) / sms * nb * kT128;
  for (int split = 2; split <= 8; split *= 2) {
    const int64_t c = (nb + split - 1) / split * kT128 + join;
    if (mt * n128 <= (split == 2 ? 75 : split == 4 ? 36 : 14) && nb >= 2 * split && c < cost) cost = c, best = {0, split, 0};
  }
  best.cost = cost;
  if (mt * n128 <= sms) return best;  // one round of 128: wider tiles take longer
  const int64_t all = (N + 255) / 256;
  for (int64_t w = all; w > 0 && (all - w) * mt <= 2 * sms; --w) {  // w tiles of 256, the rest (two rounds at most) of 128
    const int64_t rest = std::max<int64_t>(0, n128 - 2 * w) * mt, t = w * mt, full = t / sms, late = t % sms;
    // the SMs with a tile less take the first of the rest
    const int64_t early = sms - late;
    int64_t c = (full + (late ? 1 : 0)) * kT256;
    if (rest > 0) {
      const int64_t more = std::max<int64_t>(0, rest - early);
      c = std::max(c, full * kT256 + kT128);  // (a CTA of the second launch leaves once the first has ended)
      c += (more + sms - 1) / sms * kT128;
    }
    c = c * nb + (rest > 0 ? 100 : 0);  // 1 us for the second launch
    if (c < cost) cost = c, best = {(int)std::min<int64_t>(256 * w, N), 1, 0};
  }
  best.cost = cost;
  return best;
}

}  // namespace

cudaError_t linear_fp8_status_word(int32_t** word) {
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, linear_status);
  *word = static_cast<int32_t*>(p);
  return e;
}

int64_t linear_fp8_tc_cost(int T, int K, int N) { return choose(T, K, N).cost; }

const char* linear_fp8_tc_form(int T, int K, int N) {
  const TcChoice c = choose(T, K, N);
  if (c.split > 1) return c.split == 2 ? "tensor 128 split 2" : c.split == 4 ? "tensor 128 split 4" : "tensor 128 split 8";
  return c.wide == 0 ? "tensor 128" : c.wide == N ? "tensor 256" : "tensor 256 + 128";
}

cudaError_t launch_linear_fp8_tc(const LinearFp8Args& a, cudaStream_t s) {
  const TcChoice c = choose(a.T, a.K, a.N);
  if (c.split > 1) return launch_tc<128, true>(a, c.split, false, s);
  if (c.wide == 0) return launch_tc<128, false>(a, 1, false, s);
  LinearFp8Args part = a;
  part.N = c.wide;
  cudaError_t e = launch_tc<256, false>(part, 1, false, s);
  if (e != cudaSuccess || c.wide == a.N) return e;
  part.N = a.N - c.wide;
  part.w += (int64_t)c.wide * a.K;
  part.ws += (int64_t)(c.wide / kBlk) * blocks128(a.K);
  part.out = static_cast<uint8_t*>(a.out) + (int64_t)c.wide * (a.out_fp32 ? 4 : 2);
  return launch_tc<128, false>(part, 1, true, s);
}

}  // namespace fp4moe
