// Attention of many rows over the paged cache (chunks of prompts) on the
// 5th-generation tensor cores: S = Q K^T and O += P V with fp32 sums in tensor
// memory. The multiplications are the bound.
//
// A unit is 256 rows (128 for D = 256) of one KV head: two M = 128 tiles, each
// with its own S and O in tensor memory, so that one tile's softmax runs
// while the tensor cores work on the other (for D = 256 one tile with two S).
// Roles of a CTA, one per SM:
//
//   warps 0-7   softmax, a thread a row: S from tensor memory in two passes
//               (the maximum; the weights, which go back as fp16 over S as
//               the A operand of P V), the sums of weights, and the
//               epilogue. O is only rescaled when a row's maximum rises by
//               more than 2^8 over the one in use: weights up to 2^8 have the
//               same relative precision in fp16.
//   warps 8-11  loaders: quantised pages come in by plain 16-byte loads one
//               tile ahead, become the integers (u - z), exact in fp16, and go
//               to shared memory in the MMA's 128-byte swizzle; fp16 pages
//               come by TMA. Dequantising once per tile serves 256 rows. The
//               groups' scales stay in fp32 beside the tile and multiply S's
//               columns (K) and the weights (V) in the softmax: rounding
//               (u - z) s to fp16 here instead would be one rounding more per
//               cached value. Slots past the end are zeros.
//   warp 12     issues the MMAs.
//
// K is K-major (tokens x 64 dims per 128-byte swizzled row); V has the same
// layout and is the MN-major B operand, so nothing is transposed.
#pragma once

#include <algorithm>
#include <mutex>

#include "exq_attn_split.cuh"

namespace exq {
namespace chunk {

constexpr int kSoftmaxThreads = 256;
constexpr int kLoaderThreads = 128;
constexpr int kThreads = kSoftmaxThreads + kLoaderThreads + 32;
constexpr int kMmaWarp = 12;

template <int B, int D>
struct Cfg {
  static constexpr int kStreams = D == 256 ? 1 : 2;  // M = 128 tiles of a unit
  static constexpr int kRows = 128 * kStreams;
  static constexpr int kTile = D == 256 ? 64 : 128;  // cached tokens
  static constexpr int kSBufs = 2;                   // S buffers: one a stream, or two of the one stream
  static constexpr int kSlabs = D / 64;              // 64 dims: one 128-byte swizzled row
  static constexpr int kArray = kTile * D * 2;       // K or V of a stage, fp16
  static constexpr int kOffV = 0;                    // two stages each
  static constexpr int kOffK = 2 * kArray;
  static constexpr int kOffQ = 4 * kArray;
  static constexpr int kOffScale = kOffQ + kRows * D * 2;              // [stage][sk, sv][kTile] fp32
  static constexpr int kOffBar = kOffScale + 2 * 2 * kTile * 4 + 2 * 16;  // and [stage][4] of V's exponents
  static constexpr int kSmem = 1024 + kOffBar + 512;
  static constexpr int kFloats = kRows * (D + 2);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // tensor memory columns
  static constexpr int kTmemS = 0;                   // kSBufs x kTile
  static constexpr int kTmemO = 256;                 // kStreams x D
};

struct Maps {
  CUtensorMap k, v;  // fp16 pages only
};

struct Extra {
  float scale;       // |scale| log2(e); 0 is passed as 2^-126
  int negate;        // scale < 0: the MMA negates Q
};

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// shared-memory descriptor, 128-byte swizzle: `lead` is the stride between
// 64-value slabs of an MN-major operand, 1024 that between groups of 8 rows
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// instruction descriptor: fp16 A and B, fp32 D, M = 128
__device__ __forceinline__ uint32_t instr_desc(int n, bool b_mn_major, bool negate_a) {
  return (1u << 4) | (negate_a ? 1u << 13 : 0u) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (8u << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// the wait names the registers, so that no use of them moves above it
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two fp32 at a time
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// byte offset of the 16-byte chunk of dims [8 ch, 8 ch + 8) of row `row` in an
// operand of `rows` rows: 64-dim slabs of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t operand_at(int rows, int row, int ch) {
  return (ch >> 3) * (rows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); }

// ---- loaders of quantised pages: an item is the codes of one 12- or 16-byte
// piece of a token's row; consecutive threads hold 8 tokens of one piece, so
// that their 16-byte stores fall on different banks
template <int B, int D>
struct Item {
  static constexpr int kWords = B == 6 ? 3 : 4;
  static constexpr int kCodes = kWords * 32 / B;            // 32 or 16
  static constexpr int kPerRow = D / kCodes;
  static constexpr int kItems = Cfg<B, D>::kTile * kPerRow / kLoaderThreads;
};

template <int B, int D>
__device__ __forceinline__ int item_token(int it, int tid) {
  const int i = it * kLoaderThreads + tid;
  return (i & 7) + 8 * (i / (8 * Item<B, D>::kPerRow));
}
template <int B, int D>
__device__ __forceinline__ int item_piece(int it, int tid) {
  return ((it * kLoaderThreads + tid) >> 3) % Item<B, D>::kPerRow;
}

template <int B, int D>
__device__ __forceinline__ void load_items(const AttnArgs& a, int which, const int (&pages)[Item<B, D>::kItems], int head,
                                           int t, int tid, uint32_t (&w)[Item<B, D>::kItems][Item<B, D>::kWords]) {
  using I = Item<B, D>;
#pragma unroll
  for (int it = 0; it < I::kItems; ++it) {
#pragma unroll
    for (int j = 0; j < I::kWords; ++j) w[it][j] = 0;
    if (pages[it] < 0) continue;
    const int slot = (t * Cfg<B, D>::kTile + item_token<B, D>(it, tid)) & (a.page_size - 1);
    const long long g = (static_cast<long long>(pages[it]) * a.n_kv_heads + head) * a.page_size + slot;
    const uint32_t* src = a.codes[which] + g * (D * B / 32) + item_piece<B, D>(it, tid) * I::kWords;
    if constexpr (B == 6) {
#pragma unroll
      for (int j = 0; j < 3; ++j) w[it][j] = __ldg(src + j);
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
      w[it][0] = v.x, w[it][1] = v.y, w[it][2] = v.z, w[it][3] = v.w;
    }
  }
}

// Each 8 codes become a 16-byte chunk of (u - z): Q8 in the dims' order, Q4
// and Q6 as the unpackers' pairs (0 4 1 5 2 6 3 7), the order in which Q is
// loaded and O stored
template <int B, int D>
__device__ __forceinline__ void store_items(uint32_t base, int tid, const uint32_t (&w)[Item<B, D>::kItems][Item<B, D>::kWords]) {
  using I = Item<B, D>;
#pragma unroll
  for (int it = 0; it < I::kItems; ++it) {
    const int row = item_token<B, D>(it, tid), ch = item_piece<B, D>(it, tid) * (I::kCodes / 8);
#pragma unroll
    for (int j = 0; j < I::kCodes / 8; ++j) {
      uint32_t v[4];
      if constexpr (B == 4) {
        unpack8<4>(w[it][j], 0u, v);
      } else if constexpr (B == 8) {
        v[0] = split::q8_pair(w[it][2 * j], 0x4140), v[1] = split::q8_pair(w[it][2 * j], 0x4342);
        v[2] = split::q8_pair(w[it][2 * j + 1], 0x4140), v[3] = split::q8_pair(w[it][2 * j + 1], 0x4342);
      } else {
        if (j == 0) unpack8<6>(w[it][0], w[it][1], v);
        else unpack8<6>(fshr(w[it][1], w[it][2], 16), w[it][2] >> 16, v);
      }
      sts128(base + operand_at(Cfg<B, D>::kTile, row, ch + j), v[0], v[1], v[2], v[3]);
    }
  }
}

struct Phase {  // a ring position of two stages, or the parity of one barrier
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    st ^= 1;
    if (st == 0) ph ^= 1;
  }
};

template <int B, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, const __grid_constant__ Extra x) {
  using C = Cfg<B, D>;
  constexpr bool kQuant = B != 16;
  constexpr bool kPairs = B == 4 || B == 6;  // dims in the unpackers' order
  constexpr int T = C::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + C::kOffScale);
  int* exps = reinterpret_cast<int*>(scales + 4 * T);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  // barriers
  const uint32_t k_full = smem_u32(bars), k_empty = k_full + 16, v_full = k_full + 32, v_empty = k_full + 48,
                 s_full = k_full + 64, p_full = k_full + 80, o_full = k_full + 96 /* one a stream */, q_full = k_full + 112,
                 q_empty = k_full + 120, k_tma = k_full + 128, v_tma = k_full + 144, drain = k_full + 160,
                 pv_done = k_full + 168;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 22);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 23);
  int* is_last = reinterpret_cast<int*>(bars + 24);
  long long* scratch = reinterpret_cast<long long*>(smem);  // before the first tile

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, kQuant ? kLoaderThreads : 1);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, kLoaderThreads);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_full + 8 * i, 1);
      mbar_init(k_tma + 8 * i, 1);
      mbar_init(v_tma + 8 * i, 1);
    }
    mbar_init(q_full, kLoaderThreads);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    mbar_init(pv_done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  AttnWalk walk;
  walk.s = attn_share<C::kRows, T>(a, scratch);
  if (walk.s.begin >= walk.s.end) return;  // the whole CTA
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  walk.at = walk.s.begin;
  walk.pair = walk.s.pair;
  walk.pair_start = walk.s.pair_start;
  AttnPiece p;

  if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t id_qk = instr_desc(T, false, x.negate != 0), id_pv = instr_desc(D, true, false);
      Phase kr, vr;                       // ring positions of the next QK and PV
      uint32_t p_ph[2] = {0, 0}, q_ph = 0;
      const auto qk = [&](int s, int buf) {  // S = Q K^T, to buffer `buf`
        const uint32_t qa = sbase + C::kOffQ + s * (128 * D * 2), ka = sbase + C::kOffK + kr.st * C::kArray;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + C::kTmemS + buf * T, smem_desc(qa + (i >> 2) * (128 * 128) + (i & 3) * 32, 16),
                 smem_desc(ka + (i >> 2) * (T * 128) + (i & 3) * 32, 16), id_qk, i > 0);
        tc_commit(s_full + 8 * buf);
      };
      const auto pv = [&](int s, int buf, bool first) {  // O += P V
        const uint32_t va = sbase + C::kOffV + vr.st * C::kArray;
#pragma unroll
        for (int i = 0; i < T / 16; ++i)
          mma_ts(tmem + C::kTmemO + s * D, tmem + C::kTmemS + buf * T + 8 * i, smem_desc(va + i * 2048, T * 128), id_pv,
                 !(first && i == 0));
      };
      bool ok = true;
      while (ok && attn_next<C::kRows, T>(a, walk, p)) {
        const int n = p.t1 - p.t0, ns = p.u.rows > 128 ? C::kStreams : 1;
        ok = mbar_wait(q_full, q_ph, abort_flag, a);
        q_ph ^= 1;
        if (!ok) break;
        tc_after();
        if constexpr (C::kStreams == 2) {
          ok = mbar_wait(k_full + 8 * kr.st, kr.ph, abort_flag, a);
          if (!ok) break;
          tc_after();
          for (int s = 0; s < ns; ++s) qk(s, s);
          tc_commit(k_empty + 8 * kr.st);
          kr.next();
          if (n == 1) tc_commit(q_empty);
          for (int j = 0; j < n && ok; ++j) {
            for (int s = 0; s < ns && ok; ++s) {
              ok = mbar_wait(p_full + 8 * s, p_ph[s], abort_flag, a);
              p_ph[s] ^= 1;
              if (ok && s == 0) ok = mbar_wait(v_full + 8 * vr.st, vr.ph, abort_flag, a);
              if (!ok) break;
              tc_after();
              pv(s, s, j == 0);
              if (s == ns - 1) tc_commit(v_empty + 8 * vr.st);
              if (j + 1 < n) {
                if (s == 0) ok = mbar_wait(k_full + 8 * kr.st, kr.ph, abort_flag, a);
                if (!ok) break;
                tc_after();
                qk(s, s);
                if (s == ns - 1) {
                  tc_commit(k_empty + 8 * kr.st);
                  kr.next();
                  if (j + 2 == n) tc_commit(q_empty);
                }
              } else {
                tc_commit(o_full + 8 * s);
              }
            }
            vr.next();
          }
        } else {
          for (int j = 0; j < n + 1 && ok; ++j) {  // QK of tile j, then PV of tile j - 1
            if (j < n) {
              ok = mbar_wait(k_full + 8 * kr.st, kr.ph, abort_flag, a);
              if (!ok) break;
              tc_after();
              qk(0, j & 1);  // its P was read by PV of tile j - 2, issued before
              tc_commit(k_empty + 8 * kr.st);
              kr.next();
              if (j + 1 == n) tc_commit(q_empty);
            }
            if (j > 0) {
              const int buf = (j - 1) & 1;
              ok = mbar_wait(p_full + 8 * buf, p_ph[buf], abort_flag, a);
              p_ph[buf] ^= 1;
              if (ok) ok = mbar_wait(v_full + 8 * vr.st, vr.ph, abort_flag, a);
              if (!ok) break;
              tc_after();
              pv(0, buf, j == 1);
              tc_commit(v_empty + 8 * vr.st);
              vr.next();
              tc_commit(pv_done);
              if (j == n) tc_commit(o_full);
            }
          }
        }
      }
      // nothing may be in flight when tensor memory is freed
      tc_commit(drain);
      for (int r = 0; r < a.wait_limit; ++r)
        if (mbar_try_wait(drain, 0)) break;
    }
  } else if (warp >= kSoftmaxThreads / 32) {
    // -------------------------------------------------------------- loaders
    const int tid = threadIdx.x - kSoftmaxThreads;
    Phase kr, vr;
    uint32_t q_ph = 0;
    bool ok = a.starve == 0;  // test hook: the other roles' waits run out
    long long issued_k = 0, issued_v = 0;
    while (ok && attn_next<C::kRows, T>(a, walk, p)) {
      // ---- Q: [M tile][slab][128 rows][128 bytes]; rows past the unit are zeros
      ok = mbar_wait_warp(q_empty, q_ph ^ 1, abort_flag, a);
      q_ph ^= 1;
      if (!ok) break;
      const int q_rows = p.u.rows > 128 ? C::kRows : 128;
      for (int i = tid; i < q_rows * (D / 8); i += kLoaderThreads) {
        const int row = (i & 7) + 8 * (i / D), ch = (i >> 3) % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < p.u.rows) {
          int token, head;
          attn_row_of(a, p, row, token, head);
          v = __ldg(reinterpret_cast<const uint4*>(a.q.data + token * a.q.token_stride + head * a.q.head_stride + 8 * ch));
        }
        if constexpr (kPairs)
          v = make_uint4(prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632), prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
        sts128(sbase + C::kOffQ + (row >> 7) * (128 * D * 2) + operand_at(128, row & 127, ch), v.x, v.y, v.z, v.w);
      }
      async_fence();
      mbar_arrive(q_full);

      const int32_t* table = a.page_table + static_cast<long long>(p.u.b) * a.max_pages;
      const auto page_of = [&](int tok) {  // -1: zeros
        if (tok >= p.u.end) return -1;
        const int page = __ldg(table + tok / a.page_size);
        if (page < 0 || page >= a.n_pages) {
          atomicOr(a.err, kDevErrBadPage);
          return -1;
        }
        return page;
      };
      if constexpr (kQuant) {
        using I = Item<B, D>;
        // a tile ahead: page ids; a K or V ahead: codes and scales
        int pages[I::kItems], next_pages[I::kItems], spage, next_spage;
        uint32_t w[I::kItems][I::kWords];
        const int stok = tid & (T - 1);
        uint32_t scale_bits = 0;
        const auto get_pages = [&](int t, int (&pg)[I::kItems], int& sp) {
#pragma unroll
          for (int it = 0; it < I::kItems; ++it) pg[it] = t < p.t1 ? page_of(t * T + item_token<B, D>(it, tid)) : -1;
          sp = t < p.t1 ? page_of(t * T + stok) : -1;
        };
        const auto get_scale = [&](int which, int t) {
          if (spage < 0) return 0u;
          const long long g = (static_cast<long long>(spage) * a.n_kv_heads + p.head) * a.page_size +
                              ((t * T + stok) & (a.page_size - 1));
          return static_cast<uint32_t>(__ldg(a.scales[which] + g));
        };
        get_pages(p.t0, pages, spage);
        load_items<B, D>(a, 0, pages, p.head, p.t0, tid, w);
        scale_bits = get_scale(0, p.t0);
        for (int t = p.t0; t < p.t1 && ok; ++t) {
          get_pages(t + 1, next_pages, next_spage);
          // K
          ok = mbar_wait_warp(k_empty + 8 * kr.st, kr.ph ^ 1, abort_flag, a);
          if (!ok) break;
          store_items<B, D>(sbase + C::kOffK + kr.st * C::kArray, tid, w);
          // K's scales are read by the softmax of this tile, which ends
          // before V's stage of the tile is released: the V ring guards both
          ok = mbar_wait_warp(v_empty + 8 * vr.st, vr.ph ^ 1, abort_flag, a);
          if (!ok) break;
          if (tid < T) scales[(vr.st * 2) * T + stok] = half_bits_to_float(scale_bits) * x.scale;
          load_items<B, D>(a, 1, pages, p.head, t, tid, w);
          scale_bits = get_scale(1, t);
          const int e = static_cast<int>(__reduce_max_sync(0xffffffffu, scale_bits) >> 10) & 31;
          if (tid < T) scales[(vr.st * 2 + 1) * T + stok] = half_bits_to_float(scale_bits);
          if (lane == 0) exps[vr.st * 4 + (tid >> 5)] = e;
          async_fence();
          mbar_arrive(k_full + 8 * kr.st);
          kr.next();
          // V
          store_items<B, D>(sbase + C::kOffV + vr.st * C::kArray, tid, w);
#pragma unroll
          for (int it = 0; it < I::kItems; ++it) pages[it] = next_pages[it];
          spage = next_spage;
          load_items<B, D>(a, 0, pages, p.head, t + 1, tid, w);
          scale_bits = get_scale(0, t + 1);
          async_fence();
          mbar_arrive(v_full + 8 * vr.st);
          vr.next();
        }
      } else {
        const int box = min(T, a.page_size), boxes = T / box;
        int page = tid < boxes ? page_of(p.t0 * T + tid * box) : -1, last_page = -1;
        const auto issue = [&](const CUtensorMap* map, uint32_t dst, uint32_t bar, int t, int pg) {  // warp 8
          const unsigned n = __popc(__ballot_sync(0xffffffffu, pg >= 0));
          if (lane == 0) mbar_expect_tx(bar, n * box * D * 2);
          __syncwarp();
          if (pg >= 0) {
            const int slot = (t * T + lane * box) & (a.page_size - 1);
#pragma unroll
            for (int i = 0; i < C::kSlabs; ++i)
              split::tma_load_3d(dst + i * (T * 128) + lane * box * 128, map, i * 32, slot, pg * a.n_kv_heads + p.head, bar);
          }
        };
        // K of tile t, then V of tile t - 1 handed on, then V of tile t
        for (int t = p.t0; t <= p.t1 && ok; ++t) {
          if (t < p.t1) {
            ok = mbar_wait_warp(k_empty + 8 * kr.st, kr.ph ^ 1, abort_flag, a);
            if (!ok) break;
            if (tid < 32) issue(&maps.k, sbase + C::kOffK + kr.st * C::kArray, k_full + 8 * kr.st, t, page);
            ++issued_k;
            kr.next();
          }
          if (t > p.t0) {
            const int st = vr.st ^ 1;  // V of tile t - 1
            ok = mbar_wait_warp(v_tma + 8 * st, st == 0 ? vr.ph : vr.ph ^ 1, abort_flag, a);
            if (!ok) break;
            const int keep = p.u.end - (t - 1) * T;  // tokens of the tile that exist
            if (keep < T) {
              for (int i = tid; i < (T - keep) * (D / 8); i += kLoaderThreads)
                sts128(sbase + C::kOffV + st * C::kArray + operand_at(T, keep + i / (D / 8), i % (D / 8)), 0, 0, 0, 0);
              async_fence();
            }
            mbar_arrive(v_full + 8 * st);
          }
          if (t < p.t1) {
            last_page = page;
            page = tid < boxes && t + 1 < p.t1 ? page_of((t + 1) * T + tid * box) : -1;
            ok = mbar_wait_warp(v_empty + 8 * vr.st, vr.ph ^ 1, abort_flag, a);
            if (!ok) break;
            if (tid < 32) issue(&maps.v, sbase + C::kOffV + vr.st * C::kArray, v_tma + 8 * vr.st, t, last_page);
            ++issued_v;
            vr.next();
          }
        }
      }
    }
    if constexpr (!kQuant) {  // every copy lands before the CTA may go
      for (long long i = max(0ll, issued_k - 2); i < issued_k; ++i)
        for (int r = 0; r < a.wait_limit; ++r)
          if (mbar_try_wait(k_full + 8 * (i & 1), (i >> 1) & 1)) break;
      for (long long i = max(0ll, issued_v - 2); i < issued_v; ++i)
        for (int r = 0; r < a.wait_limit; ++r)
          if (mbar_try_wait(v_tma + 8 * (i & 1), (i >> 1) & 1)) break;
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int s = C::kStreams == 2 ? warp >> 2 : 0;
    const bool works = C::kStreams == 2 || warp < 4;
    const int row = s * 128 + (warp & 3) * 32 + lane;     // of the unit
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_base + C::kTmemO + s * D;
    uint32_t s_ph[2] = {0, 0}, o_ph = 0, pv_ph = 0;
    Phase sr;                                             // the scales' ring (V's)
    bool ok = true;
    while (attn_next<C::kRows, T>(a, walk, p)) {
      const bool active = works && s * 128 < p.u.rows;    // warp-uniform, the same for the stream's warps
      float m = -INFINITY, l = 0.f, base = 0.f;
      int kexp = -1;
      if (active) {
        const int rr = p.u.r0 + min(row, p.u.rows - 1), pos = p.u.len - p.u.n + rr / a.group;
        const int hi = a.causal ? min(pos + 1, p.u.len) : p.u.len, lo = a.window > 0 ? pos - a.window + 1 : 0;
        const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
        for (int t = p.t0; t < p.t1 && ok; ++t) {
          const int buf = C::kStreams == 2 ? s : (t - p.t0) & 1;
          ok = mbar_wait_warp(s_full + 8 * buf, s_ph[buf], abort_flag, a);
          s_ph[buf] ^= 1;
          if (!ok) break;
          tc_after();
          const uint32_t t_s = tmem + lane_base + C::kTmemS + buf * T;
          const float* sk = scales + sr.st * 2 * T;
          const float* sv = sk + T;
          const bool masked = t * T < all_lo || (t + 1) * T > all_hi;  // warp-uniform
          const int c_lo = lo - t * T, c_hi = hi - t * T;              // the row's columns
          // ---- maximum
          float mx = -INFINITY;
          {
            uint32_t r[2][32];
            tmem_ld32(t_s, r[0]);
#pragma unroll
            for (int c = 0; c < T / 32; ++c) {
              tmem_wait_ld(r[c & 1]);
              if (c + 1 < T / 32) tmem_ld32(t_s + 32 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                float v[4];
                if constexpr (kQuant) {
                  const float4 k4 = *reinterpret_cast<const float4*>(sk + 32 * c + i);
                  const float2 u0 = unpack_f2(mul_f2(pack_f2(__uint_as_float(r[c & 1][i]), __uint_as_float(r[c & 1][i + 1])), pack_f2(k4.x, k4.y)));
                  const float2 u1 = unpack_f2(mul_f2(pack_f2(__uint_as_float(r[c & 1][i + 2]), __uint_as_float(r[c & 1][i + 3])), pack_f2(k4.z, k4.w)));
                  v[0] = u0.x, v[1] = u0.y, v[2] = u1.x, v[3] = u1.y;
                } else {
#pragma unroll
                  for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r[c & 1][i + j]);
                }
                if (masked) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (32 * c + i + j < c_lo || 32 * c + i + j >= c_hi) v[j] = -INFINITY;
                }
                mx = fmaxf(mx, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
              }
            }
          }
          if constexpr (!kQuant) mx = mx == -INFINITY ? mx : mx * x.scale;
          // ---- the reference `base` = m - (15 - kexp): V's scales are near
          // 2^(kexp - 15), and weights times scales near 1
          int e = kexp;
          if constexpr (kQuant) {
            const int4 e4 = *reinterpret_cast<const int4*>(exps + sr.st * 4);
            const int tile_e = max(max(e4.x, e4.y), max(e4.z, e4.w));
            if (kexp < 0 || tile_e > kexp + 4) e = tile_e;
          }
          const float m1 = mx > m + 8.f ? mx : m;  // m = -inf: mx, where anything is seen
          const float shift = kQuant ? static_cast<float>(15 - e) : 0.f;
          const float base1 = (m1 == -INFINITY ? 0.f : m1) - shift;
          const bool moved = t > p.t0 && base1 != base && m != -INFINITY;  // else O is all zeros or not begun
          if constexpr (C::kStreams == 1) {
            // P V of the tile before has to be over before O is touched
            if (t > p.t0) {
              ok = mbar_wait_warp(pv_done, pv_ph, abort_flag, a);
              pv_ph ^= 1;
              if (!ok) break;
              tc_after();
            }
          }
          if (__any_sync(0xffffffffu, moved)) {
            const float f = moved ? exp2_fast(base - base1) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(t_o + 32 * c, r);
              tmem_wait_ld(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
              tmem_st32(t_o + 32 * c, r);
            }
            tmem_wait_st();
          }
          m = m1;
          kexp = e;
          base = base1;
          // ---- weights
          {
            const uint64_t nb = pack_f2(-base, -base), sc = pack_f2(x.scale, x.scale);
            uint64_t sum0 = 0, sum1 = 0;
            uint32_t r[2][32];
            tmem_ld32(t_s, r[0]);
#pragma unroll
            for (int c = 0; c < T / 32; ++c) {
              tmem_wait_ld(r[c & 1]);
              if (c + 1 < T / 32) tmem_ld32(t_s + 32 * (c + 1), r[(c + 1) & 1]);
              uint32_t out[16];
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                uint64_t u0 = pack_f2(__uint_as_float(r[c & 1][i]), __uint_as_float(r[c & 1][i + 1]));
                uint64_t u1 = pack_f2(__uint_as_float(r[c & 1][i + 2]), __uint_as_float(r[c & 1][i + 3]));
                if constexpr (kQuant) {
                  const float4 k4 = *reinterpret_cast<const float4*>(sk + 32 * c + i);
                  u0 = add_f2(mul_f2(u0, pack_f2(k4.x, k4.y)), nb);
                  u1 = add_f2(mul_f2(u1, pack_f2(k4.z, k4.w)), nb);
                } else {
                  u0 = fma_f2(u0, sc, nb);
                  u1 = fma_f2(u1, sc, nb);
                }
                const float2 f0 = unpack_f2(u0), f1 = unpack_f2(u1);
                float v[4] = {f0.x, f0.y, f1.x, f1.y};
                if (masked) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (32 * c + i + j < c_lo || 32 * c + i + j >= c_hi) v[j] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = exp2_fast(v[j]);
                u0 = pack_f2(v[0], v[1]);
                u1 = pack_f2(v[2], v[3]);
                sum0 = add_f2(sum0, u0);
                sum1 = add_f2(sum1, u1);
                if constexpr (kQuant) {
                  const float4 v4 = *reinterpret_cast<const float4*>(sv + 32 * c + i);
                  u0 = mul_f2(u0, pack_f2(v4.x, v4.y));
                  u1 = mul_f2(u1, pack_f2(v4.z, v4.w));
                }
                const float2 g0 = unpack_f2(u0), g1 = unpack_f2(u1);
                out[i / 2] = half2_bits(g0.x, g0.y);
                out[i / 2 + 1] = half2_bits(g1.x, g1.y);
              }
              tmem_st16(t_s + 16 * c, out);  // S's columns below 32 (c + 1) have been read
            }
            const float2 a0 = unpack_f2(add_f2(sum0, sum1));
            l += a0.x + a0.y;
          }
          tmem_wait_st();
          tc_before();
          mbar_arrive(p_full + 8 * buf);
          sr.next();
        }
        if (ok) {
          ok = mbar_wait_warp(o_full + 8 * s, o_ph, abort_flag, a);
          o_ph ^= 1;
          if constexpr (C::kStreams == 1) pv_ph ^= 1;  // the last P V's
          tc_after();
        }
      } else {
        // the ring of scales moves on with the other stream's tiles
        if ((p.t1 - p.t0) & 1) sr.next();
      }
      // ---- epilogue: a thread holds its row's D values
      const int c0 = p.whole ? 0 : attn_cta_of(walk.s, p.first), c1 = p.whole ? 0 : attn_cta_of(walk.s, p.first + p.u.tiles - 1);
      if (active && ok) {
        const bool has = row < p.u.rows;
        int token = 0, head = 0;
        if (has) attn_row_of(a, p, row, token, head);
        uint16_t* dst = a.out.data + token * a.out.token_stride + head * a.out.head_stride;
        float* slot = p.whole ? nullptr : attn_slot(a, blockIdx.x, static_cast<int>(blockIdx.x) == c0, C::kFloats);
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(t_o + 32 * c, r);
          tmem_wait_ld(r);
          if (has) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              // 0 4 1 5 2 6 3 7 back to the dims' order
              const int at = kPairs ? (j < 4 ? 2 * j : 2 * (j - 4) + 1) : j;
              y[j] = l > 0.f ? __uint_as_float(r[i + at]) : 0.f;
            }
            if (p.whole) {
              uint4 o;
              o.x = half2_bits(y[0] * inv, y[1] * inv);
              o.y = half2_bits(y[2] * inv, y[3] * inv);
              o.z = half2_bits(y[4] * inv, y[5] * inv);
              o.w = half2_bits(y[6] * inv, y[7] * inv);
              *reinterpret_cast<uint4*>(dst + 32 * c + i) = o;
            } else {
              float4* at = reinterpret_cast<float4*>(slot + row * D + 32 * c + i);
              at[0] = make_float4(y[0], y[1], y[2], y[3]);
              at[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
          }
          __syncwarp();
        }
        if (has) {
          if (p.whole)
            attn_store_lse(a, token, head, base, l);
          else
            slot[C::kRows * D + row] = base, slot[C::kRows * D + C::kRows + row] = l;
        }
        tc_before();  // the next unit's first P V, ordered by p_full, overwrites O
      }
      if (!p.whole) {
        __threadfence();
        softmax_sync();
        if (threadIdx.x == 0) {
          const int last = atomicAdd(a.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
          if (last) a.counters[c0] = 0u;
          *is_last = last;
        }
        softmax_sync();
        if (*is_last) {
          __threadfence();
          attn_join<C::kRows, D>(a, p, c0, c1, threadIdx.x, kSoftmaxThreads);
        }
        softmax_sync();
      }
    }
  }

  tc_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------- host

template <int B, int D>
exq_status launch(const AttnCall& call, const AttnArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<B, D>;
  Maps maps{};
  if constexpr (B == 16) {
    if (!split::encode_cache(&maps.k, a.codes[0], *call.cache, 32, CU_TENSOR_MAP_SWIZZLE_128B, C::kTile) ||
        !split::encode_cache(&maps.v, a.codes[1], *call.cache, 32, CU_TENSOR_MAP_SWIZZLE_128B, C::kTile))
      return EXQ_ERR_CUDA;
  }
  const Extra x{std::fmax(std::fabs(a.scale_log2), 0x1p-126f), a.scale_log2 < 0};
  auto fn = attn_chunk_kernel<B, D>;
  static std::once_flag once;
  std::call_once(once, [&] { cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  fn<<<std::min(sms, kAttnMaxCtas), kThreads, C::kSmem, stream>>>(maps, a, x);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

template <int B>
exq_status launch_bits(const AttnCall& call, AttnArgs& a, int sms, cudaStream_t stream) {
  switch (call.cache->D) {
    case 64: return launch<B, 64>(call, a, sms, stream);
    case 128: return launch<B, 128>(call, a, sms, stream);
    default: return launch<B, 256>(call, a, sms, stream);
  }
}

inline int rows_of(int D) { return D == 256 ? 128 : 256; }

}  // namespace chunk

exq_status launch_attn_chunk4(const AttnCall& c, AttnArgs& a, int sms, cudaStream_t stream);
exq_status launch_attn_chunk6(const AttnCall& c, AttnArgs& a, int sms, cudaStream_t stream);
exq_status launch_attn_chunk8(const AttnCall& c, AttnArgs& a, int sms, cudaStream_t stream);
exq_status launch_attn_chunk16(const AttnCall& c, AttnArgs& a, int sms, cudaStream_t stream);

}  // namespace exq
