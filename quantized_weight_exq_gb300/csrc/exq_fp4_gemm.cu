// Product of two matrices of the microscaled 4-bit format on the block-scaled
// tcgen05 tensor cores:
//   y[m][n] = fp16(f sum_k a[m][k] w[n][k]),   f = a.factor * w.factor.
//
// A pair of CTAs (a cluster of two, cta_group::2) computes 256 x 256 of y, 256
// k at a time: each CTA holds 128 rows of both operands, so that a stage is 38
// KB where one CTA's 128 x 256 would take 54 for half the work; the copies from
// L2 were that kernel's bound (220 us at 2048 x 28672 x 8192). The pairs stay
// and take tile after tile.
//
//   warp 0      brings the codes (128-byte rows, 128-byte swizzle),
//   warp 18     the scale tiles as they lie in memory (512 bytes for 128 rows x
//               4 blocks): one warp that issues all five copies of a stage is
//               slower than the MMAs.
//   warps 2-9   write the scales to tensor memory, a place for each stage, four
//               warps every second one. The tensor core's own copy
//               (tcgen05.cp) does not do here: one takes 55 clocks whatever its
//               size, the 12 of a stage 660, the four MMAs 512. From registers
//               a stage takes four warps 320, from barrier to barrier 500.
//   warp 1      of the pair's first CTA: four MMAs (K = 64) a stage, fp32 sums
//               in the tensor memory of both CTAs.
//   warps 10-17 epilogue: 32 rows x 128 columns each. The sums fill half of
//               tensor memory and the scales a part of the rest, so there is
//               one set of sums only: the warps take theirs as packed fp16 into
//               registers at once, let the next tile's MMAs begin, and store
//               while those run.
//
// Up to 128 rows of a change places with w: a CTA alone has 128 of its rows and
// all of a's as the MMA's N (16 .. 128 columns). The product is then bound by
// the codes of w: single MMAs of few columns take 46 clocks, a pair's 128
// however few (64 x 8192 x 8192 took 15 us by pairs). Where tiles are fewer
// than the SMs a cluster of two to eight CTAs divides a tile's k: each leaves
// its sums in its shared memory, where its MMAs' operands were, and each adds
// some columns of all, in order of k.
//
// The launch may begin while the one before it ends (its set-up takes 1 us):
// nothing is read or written before griddepcontrol.wait.
//
// 2048 x 28672 x 8192: E4M3 149 us (6.5 PFLOPS), E8M0 143, in runs of some 20 ms;
// after a second of nothing else the power limit has the SMs at 1.63 GHz, and E4M3
// takes 164. 1777 x 11008 x 4096 36 us (with the quantiser of a). Bound by what an SM takes in: 38 KB for 512
// clocks of MMAs are 74 bytes a clock, and copies alone reach 54 to 56. (A
// quarter of the codes brought by multicast inside the pair: 2 % less time.)
#include <algorithm>
#include <cstring>

#include "exq_fp4.cuh"

namespace exq {
namespace {

__device__ unsigned g_fp4_gemm_err;

constexpr int kTile = 256;   // rows and columns of a pair's tile
constexpr int BK = 256;      // k of a stage: four MMAs
constexpr int kThreads = 19 * 32;

constexpr int kCodes = 128 * BK / 2;  // of 128 rows
constexpr int kScaleTiles = 2048;     // the scale tiles of 128 rows x 256 k: 4 (E4M3) or 2 (E8M0)
constexpr int kRing = 5 * (2 * kCodes + 3 * kScaleTiles);
constexpr int kSmemBytes = kRing + 1024 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

// Tensor memory: the sums, then the scales of each stage (the MMA's A: 4 columns
// a tile, B: 8, or 4 for up to 128 rows). With two places for five stages the
// way from one stage's MMAs over the warps that write scales to another's
// took 1 us.
constexpr uint32_t kTmemCols = 512;
// SWAP: a's rows are the MMA's N; one CTA has a tile, not two
__host__ __device__ constexpr uint32_t scales_at(bool swap) { return swap ? 128 : 256; }
__host__ __device__ constexpr uint32_t scale_cols(bool swap) { return swap ? 32 : 48; }
__host__ __device__ constexpr int most_stages(bool swap) { return swap ? 10 : 5; }
constexpr int kMaxStages = most_stages(true);
static_assert(scales_at(false) + most_stages(false) * scale_cols(false) <= kTmemCols, "tensor memory budget");
static_assert(scales_at(true) + most_stages(true) * scale_cols(true) <= kTmemCols, "tensor memory budget");

// One stage of a CTA: 128 rows of A, B's rows or its half of them, A's scale tiles, all of B's.
struct Stage {
  int b_rows, bytes, n;
  __host__ __device__ constexpr int off_sa() const { return kCodes + b_rows * (BK / 2); }
  __host__ __device__ constexpr int off_sb() const { return off_sa() + kScaleTiles; }
};
__host__ __device__ constexpr Stage stage_of(bool swap, int n_columns) {
  Stage s{};
  s.b_rows = swap ? n_columns : n_columns / 2;
  s.bytes = s.off_sb() + (swap ? 1 : 2) * kScaleTiles;
  s.n = kRing / s.bytes < most_stages(swap) ? kRing / s.bytes : most_stages(swap);
  return s;
}
static_assert(stage_of(false, 256).n == 5 && stage_of(false, 256).bytes % 1024 == 0 && stage_of(true, 16).bytes % 1024 == 0, "stages");

struct Args {
  const uint8_t *sa, *sb;  // scale tiles of the MMA's A and B
  uint16_t* y;
  float factor;
  int A, B, K;             // rows of both
  int a_tiles, b_tiles;    // tiles of 128 rows
  int k_tiles;             // scale tiles along K
  int k_units;
  int a_rows, n_tiles;     // tiles of A (of 256 rows, SWAP: 128), and of the product in all
  int n_columns;           // of a tile: 256, or (SWAP) all of B, rounded up to 16
  int split;               // SWAP: CTAs (a cluster) that have a share of a tile's k each
  int whole_sectors;       // y's rows begin on 32-byte boundaries
  int wait_limit, starve;
};

// shared-memory descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t codes_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// instruction descriptor of the block-scaled kinds: e2m1 operands, K-major, m x n
__host__ __device__ constexpr uint32_t idesc_of(int fmt, int m, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((fmt == EXQ_FP4_E8M0 ? 1u : 0u) << 23) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// CTAS: how many work on one tile
template <int FMT, int CTAS>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                           uint32_t accumulate) {
#define EXQ_MMA(ctas, kind)                                                                                         \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                    \
               "tcgen05.mma.cta_group::" ctas ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),     \
               "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                        \
               : "memory")
  if constexpr (FMT == EXQ_FP4_E4M3 && CTAS == 2) EXQ_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (FMT == EXQ_FP4_E4M3) EXQ_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (CTAS == 2) EXQ_MMA("2", "mxf4.block_scale.scale_vec::2X");
  else EXQ_MMA("1", "mxf4.block_scale.scale_vec::2X");
#undef EXQ_MMA
}

// arrives at the barrier, in both CTAs of a pair (mask 3), when the MMAs issued so far are over
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t bar, uint16_t mask = 3) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"(mask) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Arrives at the first CTA's barrier. What it tells of lies in tensor memory
// (finished with, by a wait and a fence of tcgen05's own) or was brought to
// shared memory by copies that a barrier has seen: no ordinary store has to be
// ordered before it, and a release to the whole cluster, which drains them,
// made the product more than twice as slow (367 us, 170 without).
template <int CTAS>
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  if constexpr (CTAS == 1) return mbar_arrive(bar);
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(bar) : "memory");
}

// four fp32 numbers at this address of the cluster's CTA `rank` (several loads are to be on their way: no memory clobber)
__device__ __forceinline__ float4 peer_load(uint32_t addr, int rank) {
  float4 v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank));
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// four scale tiles (16 bytes of each for the lane) to 16 columns of this warp's lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint4 (&t)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(t[0].x), "r"(t[0].y), "r"(t[0].z), "r"(t[0].w), "r"(t[1].x), "r"(t[1].y), "r"(t[1].z), "r"(t[1].w),
        "r"(t[2].x), "r"(t[2].y), "r"(t[2].z), "r"(t[2].w), "r"(t[3].x), "r"(t[3].y), "r"(t[3].z), "r"(t[3].w)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct Turn {  // counts stages, and the parity of their barriers
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      parity ^= 1u;
    }
  }
};

template <int FMT, bool SWAP>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ Args p) {
  constexpr int kTilesUnit = BK / fp4_tile_k(FMT);
  constexpr int CTAS = SWAP ? 1 : 2;
  constexpr int kARows = 128 * CTAS;  // of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing);
  uint64_t* empty = full + kMaxStages;
  uint64_t* ready = empty + kMaxStages;  // the first CTA's: a stage's codes and scales are there in both
  uint64_t* dfull = ready + kMaxStages;
  uint64_t* dempty = dfull + 1;          // the first CTA's
  uint64_t* done = dempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % CTAS, per_tile = SWAP ? p.split : CTAS;
  const int pair = blockIdx.x / per_tile, pairs = gridDim.x / per_tile;
  const int share = SWAP ? blockIdx.x % per_tile : 0;
  const int u0 = SWAP ? share * p.k_units / p.split : 0, u1 = SWAP ? (share + 1) * p.k_units / p.split : p.k_units;
  const int n_columns = SWAP ? p.n_columns : kTile;
  const Stage stage = SWAP ? stage_of(true, n_columns) : stage_of(false, kTile);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&full[s]), 2);  // codes and scales
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&ready[s]), 4 * CTAS);
    }
    mbar_init(smem_u32(dfull), 1);
    mbar_init(smem_u32(dempty), 8 * CTAS);
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && elect_one()) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ma)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mb)) : "memory");
  }
  if (warp == 1) {
    if constexpr (CTAS == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(kTmemCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ codes
    const bool leader = elect_one();
    int issued = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!p.starve) {  // test hook: starved producers issue nothing
      Turn turn;
      bool ok = true;
      for (int t = pair; t < p.n_tiles && ok; t += pairs) {
        const int bt = t / p.a_rows, at = t - bt * p.a_rows;
        const int a_row = at * kARows + rank * 128, b_row = bt * kTile + rank * stage.b_rows;
        for (int u = u0; u < u1; ++u) {
          if (!mbar_wait_warp(smem_u32(&empty[turn.i]), turn.parity ^ 1u, abort_flag, p.wait_limit, &g_fp4_gemm_err)) {
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t st = smem_u32(smem) + turn.i * stage.bytes, bar = smem_u32(&full[turn.i]);
            mbar_expect_tx(bar, kCodes + stage.b_rows * (BK / 2));
            tma_load_2d(st, &ma, u * (BK / 2), a_row, bar);
            tma_load_2d(st + kCodes, &mb, u * (BK / 2), b_row, bar);
          }
          __syncwarp();
          turn.next(stage.n);
          ++issued;
        }
      }
    }
    await_issued(full, issued, stage.n, p.wait_limit);
  } else if (warp == 18) {
    // ------------------------------------------------------------ scales
    const bool leader = elect_one();
    int issued = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!p.starve) {
      Turn turn;
      bool ok = true;
      for (int t = pair; t < p.n_tiles && ok; t += pairs) {
        const int bt = t / p.a_rows, at = t - bt * p.a_rows;
        const int a_tile = CTAS * at + rank, b_parts = SWAP ? 1 : min(2, p.b_tiles - 2 * bt);
        const bool has_a = a_tile < p.a_tiles;  // (else the rows are past the matrix: zero codes, any scales)
        const uint8_t* sa = p.sa + static_cast<size_t>(a_tile) * p.k_tiles * 512;
        const uint8_t* sb = p.sb + static_cast<size_t>(2 * bt) * p.k_tiles * 512;
        const uint8_t* sb2 = sb + static_cast<size_t>(p.k_tiles) * 512;
        if constexpr (SWAP) {
          sa += static_cast<size_t>(u0) * kTilesUnit * 512;
          sb += static_cast<size_t>(u0) * kTilesUnit * 512;
        }
        for (int u = u0; u < u1; ++u) {
          if (!mbar_wait_warp(smem_u32(&empty[turn.i]), turn.parity ^ 1u, abort_flag, p.wait_limit, &g_fp4_gemm_err)) {
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t st = smem_u32(smem) + turn.i * stage.bytes, bar = smem_u32(&full[turn.i]);
            const uint32_t bytes = min(kTilesUnit, p.k_tiles - u * kTilesUnit) * 512;
            mbar_expect_tx(bar, ((has_a ? 1 : 0) + b_parts) * bytes);
            if (has_a) bulk_load(st + stage.off_sa(), sa, bytes, bar);
            bulk_load(st + stage.off_sb(), sb, bytes, bar);
            if (!SWAP && b_parts == 2) bulk_load(st + stage.off_sb() + kScaleTiles, sb2, bytes, bar);
          }
          sa += kTilesUnit * 512;
          sb += kTilesUnit * 512;
          sb2 += kTilesUnit * 512;
          __syncwarp();
          turn.next(stage.n);
          ++issued;
        }
      }
    }
    await_issued(full, issued, stage.n, p.wait_limit);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs, by the first CTA
    if (rank == 0) {
      const bool leader = elect_one();
      const uint32_t idesc = idesc_of(FMT, kARows, n_columns);
      constexpr uint32_t kTileColsB = SWAP ? 4 : 8;
      Turn turn;
      uint32_t tile_parity = 1;
      bool ok = true;
      for (int t = pair; t < p.n_tiles && ok; t += pairs) {
        if (!mbar_wait_warp(smem_u32(dempty), tile_parity, abort_flag, p.wait_limit, &g_fp4_gemm_err)) break;
        tile_parity ^= 1u;
        tc_fence_after();
        for (int u = u0; u < u1; ++u) {
          if (!mbar_wait_warp(smem_u32(&ready[turn.i]), turn.parity, abort_flag, p.wait_limit, &g_fp4_gemm_err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + turn.i * stage.bytes;
          const uint32_t sa = tmem + scales_at(SWAP) + turn.i * scale_cols(SWAP), sb = sa + 16;
          const int n_k = min(4, (p.K - u * BK + 63) / 64);  // MMAs with k of the matrices
          if (leader) {
            const uint64_t ad = codes_desc(st), bd = codes_desc(st + kCodes);
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 64 k: 32 bytes of a row
              if (j >= n_k) break;
              if constexpr (FMT == EXQ_FP4_E4M3)
                mma_scaled<FMT, CTAS>(tmem, ad + 2 * j, bd + 2 * j, idesc, sa + 4 * j, sb + kTileColsB * j, u != u0 || j != 0);
              else  // two scales of the tile's four: byte 0 or 2 of each word
                mma_scaled<FMT, CTAS>(tmem, ad + 2 * j, bd + 2 * j, (j & 1) ? idesc | (2u << 4) | (2u << 29) : idesc, sa + 4 * (j >> 1),
                              sb + kTileColsB * (j >> 1), u != u0 || j != 0);
            }
            commit<CTAS>(smem_u32(&empty[turn.i]));
          }
          __syncwarp();
          turn.next(stage.n);
        }
        if (leader) commit<CTAS>(smem_u32(dfull));
        __syncwarp();
      }
      // the MMAs are over before tensor memory is given back
      if (leader) commit<CTAS>(smem_u32(done), 1);
      __syncwarp();
      for (int r = 0; r < p.wait_limit; ++r)
        if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(done), 0))) break;
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------ scales to tensor memory
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Turn turn;
    // Stages by their place, not by their turn: four warps see every phase of the barriers they wait on. (A wait tells a
    // phase from the one before, not from the one before that, and copies may land out of order.)
    const int group = (warp - 2) >> 2;
    bool ok = true;
    for (int t = pair; t < p.n_tiles && ok; t += pairs) {
      for (int u = u0; u < u1; ++u) {
        if ((turn.i & 1) != group) {
          turn.next(stage.n);
          continue;
        }
        if (!mbar_wait_warp(smem_u32(&full[turn.i]), turn.parity, abort_flag, p.wait_limit, &g_fp4_gemm_err)) {
          ok = false;
          break;
        }
        const uint8_t* sa = smem + turn.i * stage.bytes + stage.off_sa() + lane * 16;
        const uint8_t* sb = smem + turn.i * stage.bytes + stage.off_sb() + lane * 16;
        uint4 a[4], b[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[j] = *reinterpret_cast<const uint4*>(sa + j % kTilesUnit * 512);
          if constexpr (SWAP) {
            b[0][j] = *reinterpret_cast<const uint4*>(sb + j % kTilesUnit * 512);
          } else {
            // columns: tile 0 of the first and the second 128 rows, tile 1 of both, ...
            b[0][j] = *reinterpret_cast<const uint4*>(sb + (j & 1) * kScaleTiles + (j >> 1) * 512);
            if (kTilesUnit == 4) b[1][j] = *reinterpret_cast<const uint4*>(sb + (j & 1) * kScaleTiles + (2 + (j >> 1)) * 512);
          }
        }
        tc_fence_after();
        const uint32_t to = tmem + lanes + scales_at(SWAP) + turn.i * scale_cols(SWAP);  // (the stage was free, so this is)
        tmem_st16(to, a);
        tmem_st16(to + 16, b[0]);
        if (!SWAP && kTilesUnit == 4) tmem_st16(to + 32, b[1]);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<CTAS>(smem_u32(&ready[turn.i]));
        turn.next(stage.n);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 10) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t parity = 0;
    for (int t = pair; t < p.n_tiles; t += pairs) {
      const int bt = t / p.a_rows, at = t - bt * p.a_rows;
      if (!mbar_wait_warp(smem_u32(dfull), parity, abort_flag, p.wait_limit, &g_fp4_gemm_err) || *abort_flag) break;
      parity ^= 1u;
      tc_fence_after();
      const int row = at * kARows + rank * 128 + quarter * 32 + lane;
      if constexpr (SWAP) {
        // groups of 16 columns (rows of y), the two halves of the warps in turn
        uint32_t v[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((2 * c + half) * 16 < n_columns) tmem_ld16(tmem + lanes + (2 * c + half) * 16, v[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<CTAS>(smem_u32(dempty));
        if (p.split > 1) {  // the ring is free: sums [columns][rows], for the cluster
          float* sums = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if ((2 * c + half) * 16 < n_columns) sums[((2 * c + half) * 16 + j) * 128] = __uint_as_float(v[c][j]);
        } else if (row < p.A) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int m0 = (2 * c + half) * 16;
            uint16_t* dst = p.y + static_cast<size_t>(m0) * p.A + row;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (m0 + j < p.B) *dst = __half_as_ushort(__float2half_rn(__uint_as_float(v[c][j]) * p.factor));
              dst += p.A;
            }
          }
        }
      } else {
        uint32_t h[64];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(tmem + lanes + half * 128 + 32 * c, r);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            h[16 * c + j] = pack_half2(__uint_as_float(r[2 * j]) * p.factor, __uint_as_float(r[2 * j + 1]) * p.factor);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<CTAS>(smem_u32(dempty));
        const int n0 = bt * kTile + half * 128;
        if (row < p.A) {
          uint16_t* dst = p.y + static_cast<size_t>(row) * p.B + n0;
          if (p.whole_sectors) {  // 32 bytes at a time: a lane's stores fill sectors (with 16 they take twice as long)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (n0 + 16 * j < p.B)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * j), "r"(h[8 * j]),
                             "r"(h[8 * j + 1]), "r"(h[8 * j + 2]), "r"(h[8 * j + 3]), "r"(h[8 * j + 4]), "r"(h[8 * j + 5]),
                             "r"(h[8 * j + 6]), "r"(h[8 * j + 7]) : "memory");
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (n0 + 8 * j < p.B) *reinterpret_cast<uint4*>(dst + 8 * j) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
          }
        }
      }
    }
  }

  __syncwarp();
  if constexpr (SWAP) {
    if (p.split > 1) {
      // Each CTA adds some columns of all, in order of k; the last barrier keeps shared memory until it is read.
      cluster_sync();
      const int row = pair * 128 + 4 * lane, m0 = share * n_columns / p.split, m1 = (share + 1) * n_columns / p.split;
      if (warp >= 10 && row < p.A && !*abort_flag) {
        for (int m = m0 + warp - 10; m < min(m1, p.B); m += 32) {  // four columns at a time, every eighth one
          float4 v[4] = {};
          for (int r = 0; r < p.split; ++r) {
            float4 t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (m + 8 * i < m1) t[i] = peer_load(smem_u32(smem) + (m + 8 * i) * 512 + lane * 16, r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (m + 8 * i < m1) v[i] = make_float4(v[i].x + t[i].x, v[i].y + t[i].y, v[i].z + t[i].z, v[i].w + t[i].w);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (m + 8 * i < min(m1, p.B))
              *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(m + 8 * i) * p.A + row) =
                  make_uint2(pack_half2(v[i].x * p.factor, v[i].y * p.factor), pack_half2(v[i].z * p.factor, v[i].w * p.factor));
        }
      }
      __syncwarp();
      cluster_sync();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();  // the other CTA's tensor memory and barriers are in use until here
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CTAS == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

int div_up(int a, int b) { return (a + b - 1) / b; }

// CTAs for a tile of up to 128 rows: as many as there are SMs for, in a cluster
// (of four and eight fewer fit), with four units of k each and more, eight
// where the sums to join are many. By one CTA and by these: 64 x 8192 x 8192
// (2) 12.6 and 11.5 us, 64 x 4096 x 11008 (4) 14.4 and 10.0, 64 x 1024 x 8192
// (8) 11.5 and 7.3, 32 x 4096 x 4096 (4) 7.7 and 6.8; 128 x 4096 x 4096 8.2,
// with four 9.1.
int split_of(int n_tiles, int n_columns, int k_units, int sms) {
  const int least = n_columns > 64 ? 8 : 4;
  for (int split = 8; split > 1; split /= 2)
    if (static_cast<long long>(n_tiles) * split <= (split == 2 ? sms : split == 4 ? sms * 6 / 7 : sms * 2 / 3) && k_units >= least * split)
      return split;
  return 1;
}

}  // namespace

exq_status launch_fp4_gemm(const exq_fp4_matrix& x, const exq_fp4_matrix& w, uint16_t* y, int sms, int device,
                           cudaStream_t stream) {
  const bool swap = x.rows <= 128;
  const exq_fp4_matrix &a = swap ? w : x, &b = swap ? x : w;
  const int n_columns = swap ? div_up(x.rows, 16) * 16 : kTile;
  CUtensorMap ma, mb;
  if (!encode_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.K / 2, a.rows, a.K / 2, BK / 2, 128,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b.codes, b.K / 2, b.rows, b.K / 2, BK / 2, swap ? n_columns : kTile / 2,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B))
    return EXQ_ERR_CUDA;
  Args p{};
  p.sa = a.scales;
  p.sb = b.scales;
  p.y = y;
  p.factor = static_cast<float>(a.factor * b.factor);
  p.A = a.rows;
  p.B = b.rows;
  p.K = a.K;
  p.a_tiles = div_up(a.rows, 128);
  p.b_tiles = div_up(b.rows, 128);
  p.k_tiles = div_up(a.K, fp4_tile_k(a.format));
  p.k_units = div_up(a.K, BK);
  p.a_rows = div_up(a.rows, swap ? 128 : kTile);
  p.n_tiles = p.a_rows * div_up(b.rows, kTile);
  p.n_columns = n_columns;
  p.split = swap ? split_of(p.n_tiles, n_columns, p.k_units, sms) : 1;
  p.whole_sectors = b.rows % 16 == 0 && (reinterpret_cast<uintptr_t>(y) & 31u) == 0;
  const int starve = testing_starve_rounds();
  p.wait_limit = starve > 0 ? starve : kFp4WaitLimit;
  p.starve = starve > 0 ? 1 : 0;

  const bool e4m3 = a.format == EXQ_FP4_E4M3;
  auto fn = e4m3 ? (swap ? gemm_kernel<EXQ_FP4_E4M3, true> : gemm_kernel<EXQ_FP4_E4M3, false>)
                 : (swap ? gemm_kernel<EXQ_FP4_E8M0, true> : gemm_kernel<EXQ_FP4_E8M0, false>);
  static PerDevice attr[4];
  if (!attr[2 * e4m3 + swap].once(device, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) == cudaSuccess;
      }))
    return EXQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(swap ? std::min(p.n_tiles * p.split, sms) : 2 * std::min(p.n_tiles, std::max(sms / 2, 1)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = swap ? p.split : 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, ma, mb, p) == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

unsigned take_fp4_gemm_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_fp4_gemm_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_fp4_gemm_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
