// Attention of few rows over the paged cache (decoded tokens, drafts): HBM is
// the bound, the cache is read once, as packed codes.
//
//   S^T = K Q^T and O^T = V^T P^T on mma.sync.m16n8k16: the cache is the A
//   operand, 16 tokens (or 16 dims) a fragment, and the query rows are B's 8
//   columns, so 8 rows cost one instruction per 256 cached values.
//
// Codes become the small integers (u - z), exact in fp16, and the groups'
// scales stay outside the products, in fp32:
//   q . k_t = s_t sum_d q_d (u_td - z),   sum_t (p_t s_t) (u_td - z),
// so a pair of codes costs an AND-OR that plants them in the mantissa of 1024
// and one exact fp16x2 subtraction (and part of a shift), the same as the
// weights of the GEMV. Leaving the zero point in (multiplying by u, planted
// or as a subnormal, and subtracting z sum_t p_t s_t after) would save the
// subtraction, but the tensor cores align products by their operands'
// exponents and keep about 24 bits: for weights of mixed size the sums were
// off by up to 2^-14 of the largest.
// K and V differ in how their fragments are gathered: K's words come by
// ldmatrix as they lie; V needs two tokens' codes of one dim in a register,
// which ldmatrix.trans gives for 16-bit units of 4 (Q4), 2 (Q8) or 1 (fp16)
// values; Q6's codes straddle such units and take plain loads and byte
// permutes. The order of dims within a fragment follows the packing; Q is
// loaded, and O stored, in that order.
//
// A CTA is two pairs of warps that take the 64-token tiles in turn, each warp
// 32 tokens as two slices of 16 side by side (so that a wait and a vote serve
// 32 tokens, and the slices' chains overlap), with softmax statistics and
// sums of their own until the unit ends, and a producer warp
// that fills a ring of stages by TMA: one box per page (or 64 tokens of it),
// swizzled so that ldmatrix is free of bank conflicts, and the scales beside
// it. Slots past the last token are masked in S, and V's (fp16) zeroed.
//
// 8 KV heads of 128, 8 query heads each: one sequence of 131072 tokens Q8 (273
// MB) 61 us, 4.4 TB/s, 66 % of the copy rate; 32 ragged ones up to 8192
// Q4 (152 MB) 44 us, half of it at the copy rate, the rest unpacking, starts
// and joins; one of 500 tokens 10 us.
#pragma once

#include <algorithm>

#include "exq_attn.cuh"

namespace exq {
namespace split {

constexpr int kTile = 64;
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;

template <int B, int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = D * B / 8;
  // parts of a row as TMA boxes; 128-byte parts at most where rows are swizzled
  static constexpr int kPartBytes = B == 6 ? kRowBytes : kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kParts = kRowBytes / kPartBytes;
  static constexpr int kArray = kTile * kRowBytes;        // K or V of a stage
  static constexpr int kScale = B == 16 ? 0 : kTile * 2;  // scales of K or V
  static constexpr int kStage = ((2 * kArray + 2 * kScale + 1023) / 1024) * 1024;
  // the warps' sums meet in `regions` copies (4: one barrier, 1: four)
  static constexpr int merge_bytes(int regions) { return regions * kRows * D * 4 + 2 * kConsumers * kRows * 4; }
  static constexpr int fit(int ctas, int regions) {
    return ((227 * 1024) / ctas - 2048 - 256 - 5 * static_cast<int>(sizeof(AttnState)) - merge_bytes(regions)) / kStage;
  }
  // CTAs of an SM: as registers allow, fewer until each has 4 stages
  static constexpr int kByRegs = D * NT > 128 ? 2 : D * NT > 64 ? 3 : 4;
  static constexpr int kCtas = fit(kByRegs, 1) >= 4 ? kByRegs : kByRegs > 2 && fit(2, 1) >= 4 ? 2 : 1;
  // Two pairs of warps take tiles in turn. The stages are even in number, so
  // a stage always belongs to the same pair: a warp that met a stage only now
  // and then could take the phase before last for the last. Where 4 stages do
  // not fit (fp16, D = 256), all warps share every tile.
  static constexpr bool kAlternate = fit(kCtas, 1) >= 4;
  static constexpr int even(int n) { return n > 8 ? 8 : n & ~1; }
  static constexpr int kWide = even(fit(kCtas, kConsumers));
  static constexpr int kRegions = kAlternate && (kWide == even(fit(kCtas, 1)) || kWide >= 6) ? kConsumers : 1;
  static constexpr int kStages = kAlternate ? even(fit(kCtas, kRegions)) : fit(kCtas, kRegions);
  static constexpr int kMerge = merge_bytes(kRegions);
  static constexpr int kSlices = kAlternate ? 2 : 1;  // of 16 tokens, of a warp in a tile
  static constexpr int kSmem = 1024 + kStages * kStage + ((kMerge + 15) / 16) * 16 + 256 + 5 * sizeof(AttnState);
  static_assert(kStages >= 2 && (!kAlternate || kStages % 2 == 0), "stages");
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory");
  static constexpr int kFloats = kRows * (D + 2);
};

struct Maps {
  CUtensorMap k, v;
};

// Copies are issued by a whole warp with the same operands, one lane elected
// in the instruction: the operands stay in uniform registers. Each issued by
// some lane on its own took 200 cycles, and the producer was the bound.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
      : "memory");
}

// the same value in every lane, known as such to the compiler
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

// Byte offset of 16-byte chunk `ch` of token row `row` in a stage's K or V,
// where TMA put it: its swizzle XORs the chunk's index in a 128-, 64- or
// 32-byte row with address bits 7 and up.
template <typename C>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  constexpr int kPer = C::kPartBytes / 16;  // 8, 4 or 2
  const int part = ch / kPer, in = ch % kPer;
  const int x = kPer == 8 ? row & 7 : kPer == 4 ? (row >> 1) & 3 : (row >> 2) & 1;
  return part * (kTile * C::kPartBytes) + row * C::kPartBytes + ((in ^ x) << 4);
}

// The token of a 16-token slice at fragment index i: as they lie, except for
// Q6, whose plain loads of V then touch four neighbouring tokens at a time.
template <int B>
__device__ __forceinline__ int token_at(int i) {
  if constexpr (B == 6) return (i & 8) + ((i >> 1) & 3) + 4 * (i & 1);
  return i;
}

// (u - z) of Q8 codes planted in 1024
__device__ __forceinline__ uint32_t q8_pair(uint32_t w, uint32_t sel) {
  return hadd2(prmt(w, 0x64646464u, sel), pack2(f16_bits(-(1024 + 128)), f16_bits(-(1024 + 128))));
}

// (u_i - z) of two tokens a, b from 48 bits of Q6 codes of each
__device__ __forceinline__ void q6_two(uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t (&v)[8]) {
  const uint32_t x01 = prmt(alo, blo, 0x5410), x12 = prmt(alo, blo, 0x6521), x23 = prmt(alo, blo, 0x7632);
  const uint32_t wa = fshr(alo, ahi, 16), wb = fshr(blo, bhi, 16);
  const uint32_t y = prmt(wa, wb, 0x6521), z = prmt(wa, wb, 0x7632);
  v[0] = unbias<0, 0, 32>(and_or(x01, 0x003F003Fu, kMagic));
  v[1] = unbias<4, 4, 32>(and_or(x01 >> 2, 0x03F003F0u, kMagic));
  v[2] = unbias<4, 4, 32>(and_or(x12, 0x03F003F0u, kMagic));
  v[3] = unbias<2, 2, 32>(and_or(x23, 0x00FC00FCu, kMagic));
  v[4] = unbias<0, 0, 32>(and_or(y, 0x003F003Fu, kMagic));
  v[5] = unbias<4, 4, 32>(and_or(y >> 2, 0x03F003F0u, kMagic));
  v[6] = unbias<4, 4, 32>(and_or(z, 0x03F003F0u, kMagic));
  v[7] = unbias<2, 2, 32>(and_or(z >> 8, 0x00FC00FCu, kMagic));
}

// O's dim of (16-dim tile, half of its rows, lane group g)
template <int B, int D>
__device__ __forceinline__ int dim_of(int mt, int half, int g) {
  if constexpr (B == 4) return 32 * (mt >> 1) + 4 * g + 2 * (mt & 1) + half;
  if constexpr (B == 6) return g * (D / 8) + 2 * mt + half;
  if constexpr (B == 8) return 16 * mt + 2 * g + half;
  return 16 * mt + 8 * half + g;
}

// S^T += K Q^T of 16 tokens from row `row0` of a stage, in two chains of sums
template <int B, int D, int NT>
__device__ __forceinline__ void scores(uint32_t kbase, int row0, int lane, const uint32_t (&bq)[NT][D / 16][2],
                                       float (&s)[NT][4], float (&s2)[NT][4]) {
  using C = Cfg<B, D, NT>;
  const int g = lane >> 2, c = lane & 3;
  const int tok_a = row0 + token_at<B>(g), tok_b = row0 + token_at<B>(g + 8);
  if constexpr (B == 6) {
    constexpr int kWin = D / 32;  // 48-bit windows of a lane's D / 4 codes
    constexpr int kW = kWin * 3 / 2;
    uint32_t wa[kW], wb[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      wa[i] = lds32(kbase + tok_a * C::kRowBytes + c * (kW * 4) + 4 * i);
      wb[i] = lds32(kbase + tok_b * C::kRowBytes + c * (kW * 4) + 4 * i);
    }
#pragma unroll
    for (int i = 0; i < kWin; ++i) {
      const int w = (i / 2) * 3 + (i & 1);
      uint32_t pa[4], pb[4];
      if (i & 1) {
        unpack8<6>(fshr(wa[w], wa[w + 1], 16), wa[w + 1] >> 16, pa);
        unpack8<6>(fshr(wb[w], wb[w + 1], 16), wb[w + 1] >> 16, pb);
      } else {
        unpack8<6>(wa[w], wa[w + 1], pa);
        unpack8<6>(wb[w], wb[w + 1], pb);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma(s[nt], pa[0], pb[0], pa[1], pb[1], bq[nt][2 * i][0], bq[nt][2 * i][1]);
        mma(s2[nt], pa[2], pb[2], pa[3], pb[3], bq[nt][2 * i + 1][0], bq[nt][2 * i + 1][1]);
      }
    }
  } else {
    constexpr int kChunks = C::kRowBytes / 16;
    const int lrow = row0 + (lane & 15), lch = lane >> 4;
#pragma unroll
    for (int q = 0; q < kChunks; q += 2) {
      uint32_t r[4];
      ldsm4<false>(kbase + chunk_at<C>(lrow, q + lch), r);
      if constexpr (B == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pa[4], pb[4];
          unpack8<4>(r[2 * h], 0u, pa);
          unpack8<4>(r[2 * h + 1], 0u, pb);
          const int i = 2 * (q + h);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(s[nt], pa[0], pb[0], pa[1], pb[1], bq[nt][i][0], bq[nt][i][1]);
            mma(s2[nt], pa[2], pb[2], pa[3], pb[3], bq[nt][i + 1][0], bq[nt][i + 1][1]);
          }
        }
      } else if constexpr (B == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = r[2 * h], w1 = r[2 * h + 1];
          const uint32_t a0 = q8_pair(w0, 0x4140), a1 = q8_pair(w1, 0x4140), a2 = q8_pair(w0, 0x4342),
                         a3 = q8_pair(w1, 0x4342);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(h ? s2[nt] : s[nt], a0, a1, a2, a3, bq[nt][q + h][0], bq[nt][q + h][1]);
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma((q & 2) ? s2[nt] : s[nt], r[0], r[1], r[2], r[3], bq[nt][q / 2][0], bq[nt][q / 2][1]);
      }
    }
  }
}

// Which of a lane's fp16 values of V are to be cleaned: bits of tokens that are
// taken as they are or cleaned (`keep`), and of those that are cleaned (`some`).
struct Clean {
  uint32_t keep, some;
  __device__ __forceinline__ void two(int x, int begin, int end, int all_lo, int all_hi) {  // tokens x and x + 1
    const auto seen = [&](int t) { return t >= begin && t < end; };
    const auto shared = [&](int t) { return t >= all_lo && t < all_hi; };
    keep = (seen(x) ? 0xFFFFu : 0u) | (seen(x + 1) ? 0xFFFF0000u : 0u);
    some = keep & ((shared(x) ? 0u : 0x8000u) | (shared(x + 1) ? 0u : 0x80000000u));
  }
  __device__ __forceinline__ void apply(uint32_t& v, bool& taken) const {
    v &= keep;
    const uint32_t out = attn_not_finite(v, some);
    v &= ~out;
    taken |= out != 0;
  }
};

// O^T += V^T P^T of the same; fp16 values of tokens c, c + 1 (a) and c + 8, c + 9 (b) are cleaned where `clean` says so
template <int B, int D, int NT>
__device__ __forceinline__ void values(uint32_t vbase, int row0, int lane, bool clean, const Clean& a, const Clean& b, bool& taken,
                                       const uint32_t (&pb)[NT][2], float (&o)[NT][D / 16][4]) {
  using C = Cfg<B, D, NT>;
  const int g = lane >> 2, c = lane & 3;
  if constexpr (B == 6) {
    // tokens (c, 4 + c) and (8 + c, 12 + c) of the slice, D / 8 codes from dim g D / 8
    constexpr int kWin = D / 64;
    const int ta = row0 + c;
#pragma unroll
    for (int i = 0; i < kWin; ++i) {
      uint32_t w[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int bit = g * (D / 8 * 6) + 48 * i;  // of the row
        const uint32_t at = vbase + (ta + 4 * j) * C::kRowBytes + (bit >> 5) * 4;
        const uint32_t x = lds32(at), y = lds32(at + 4);
        w[j][0] = fshr(x, y, bit & 16);
        w[j][1] = y >> (bit & 16);
      }
      uint32_t va[8], vb[8];
      q6_two(w[0][0], w[0][1], w[1][0], w[1][1], va);
      q6_two(w[2][0], w[2][1], w[3][0], w[3][1], vb);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma(o[nt][4 * i + j], va[2 * j], va[2 * j + 1], vb[2 * j], vb[2 * j + 1], pb[nt][0], pb[nt][1]);
    }
  } else {
    constexpr int kChunks = C::kRowBytes / 16;
    const int lrow = row0 + (lane & 15), lch = lane >> 4;
#pragma unroll
    for (int q = 0; q < kChunks; q += 2) {
      uint32_t r[4];
      ldsm4<true>(vbase + chunk_at<C>(lrow, q + lch), r);
      if constexpr (B == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // the unpacker's pairs are here (token a, token b) of dims 4g .. 4g + 3
          uint32_t va[4], vb[4];
          unpack8<4>(r[2 * h], 0u, va);
          unpack8<4>(r[2 * h + 1], 0u, vb);
          const int i = 2 * (q + h);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(o[nt][i], va[0], va[1], vb[0], vb[1], pb[nt][0], pb[nt][1]);
            mma(o[nt][i + 1], va[2], va[3], vb[2], vb[3], pb[nt][0], pb[nt][1]);
          }
        }
      } else if constexpr (B == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w0 = r[2 * h], w1 = r[2 * h + 1];
          const uint32_t a0 = q8_pair(w0, 0x4240), a1 = q8_pair(w0, 0x4341), a2 = q8_pair(w1, 0x4240),
                         a3 = q8_pair(w1, 0x4341);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(o[nt][q + h], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      } else {
        if (clean) a.apply(r[0], taken), a.apply(r[2], taken), b.apply(r[1], taken), b.apply(r[3], taken);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(o[nt][q / 2], r[0], r[2], r[1], r[3], pb[nt][0], pb[nt][1]);
      }
    }
  }
}

template <int B, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Cfg<B, D, NT>::kCtas))
    attn_split_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a) {
  using C = Cfg<B, D, NT>;
  constexpr bool kQuant = B != 16;
  constexpr int kSteps = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
  float* stat_m = merge + C::kRegions * C::kRows * D;
  float* stat_l = stat_m + kConsumers * C::kRows;
  uint8_t* tail = smem + C::kStages * C::kStage + ((C::kMerge + 15) / 16) * 16;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kStages);
  int* is_last = const_cast<int*>(abort_flag) + 1;
  int* cleaned = is_last + 1;  // of each consumer warp: something was taken out of V in the unit

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), C::kAlternate ? kConsumers / 2 : kConsumers);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  AttnState& state = reinterpret_cast<AttnState*>(tail + 256)[warp];
  if (!attn_begin<C::kRows, kTile>(a, state)) return;  // the whole CTA
  __syncthreads();                                      // the barriers are initialised
  const AttnPiece& p = state.p;

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    if (a.starve) return;  // test hook: the consumers' waits run out
    const int box = min(kTile, a.page_size);      // tokens of a TMA box
    const int boxes = kTile / box;                // of a tile
    int st = 0;
    uint32_t ph = 0;
    long long issued = 0;
    bool ok = true;
    while (ok && attn_next<C::kRows, kTile>(a, state)) {
      const int32_t* table = a.page_table + static_cast<long long>(p.u.b) * a.max_pages;
      const int t0 = p.t0, t1 = p.t1, head = p.head, begin = p.u.begin, end = p.u.end;
      const int b0 = t0 * boxes, b1 = t1 * boxes;      // boxes of the piece
      const auto page_of = [&](int bx) {               // -1: nothing to copy
        const int tok = bx * box;
        if (bx >= b1 || tok >= end || tok + box <= begin) return -1;
        const int page = __ldg(table + tok / a.page_size);
        if (page < 0 || page >= a.n_pages) {
          atomicOr(a.err, kDevErrBadPage);
          return -1;
        }
        return page;
      };
      int have = b0, page = page_of(b0 + lane), next = page_of(b0 + 32 + lane);
      for (int t = t0; t < t1; ++t) {
        if (t * boxes >= have + 32) {
          have += 32;
          page = next;
          next = page_of(have + 32 + lane);
        }
        const int at = t * boxes - have;  // the tile's boxes are those of lanes at .. at + boxes - 1
        const unsigned there = (__ballot_sync(0xffffffffu, page >= 0) >> at) & ((1u << boxes) - 1u);
        ok = mbar_wait_warp(smem_u32(&empty[st]), ph ^ 1, abort_flag, a);
        if (!ok) break;
        const uint32_t bar = uniform(smem_u32(&full[st])), base = uniform(smem_u32(smem + st * C::kStage));
        expect_tx(bar, uniform(__popc(there) * box * (2 * C::kRowBytes + (kQuant ? 4 : 0))));
        for (int i = 0; i < boxes; ++i) {
          if (!((there >> i) & 1u)) continue;
          const int block = __shfl_sync(0xffffffffu, page, at + i) * a.n_kv_heads + head;
          const uint32_t slot = uniform((t * kTile + i * box) & (a.page_size - 1)), blk = uniform(block);
          const uint32_t off = base + uniform(i * box) * C::kPartBytes;
#pragma unroll
          for (int k = 0; k < C::kParts; ++k) {
            tma_load_3d(off + k * (kTile * C::kPartBytes), &maps.k, k * (C::kPartBytes / 4), slot, blk, bar);
            tma_load_3d(off + C::kArray + k * (kTile * C::kPartBytes), &maps.v, k * (C::kPartBytes / 4), slot, blk, bar);
          }
          if constexpr (kQuant) {
            const long long grp = static_cast<long long>(blk) * a.page_size + slot;
            const uint32_t sc = base + 2 * C::kArray + uniform(i * box) * 2;
            bulk_load(sc, a.scales[0] + grp, box * 2, bar);
            bulk_load(sc + C::kScale, a.scales[1] + grp, box * 2, bar);
          }
        }
        ++issued;
        if (++st == C::kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    // every stage's copies land before the CTA may go
    for (long long i = max(0ll, issued - C::kStages); i < issued; ++i)
      for (int r = 0; r < a.wait_limit; ++r)
        if (mbar_try_wait(smem_u32(&full[i % C::kStages]), (i / C::kStages) & 1)) break;
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  constexpr int kSlices = C::kSlices;
  const int row0 = C::kAlternate ? (warp & 1) * 32 : warp * 16;  // the warp's tokens in a tile
  const int turn = warp >> 1;                                    // its pair's tiles: even or odd ones of the CTA's
  int st = 0, tile = 0;
  uint32_t ph = 0;
  while (attn_next<C::kRows, kTile>(a, state)) {
    const int t0 = p.t0, t1 = p.t1, begin = p.u.begin, end = p.u.end;
    // Q as B fragments: column g of tile nt is row 8 nt + g
    uint32_t bq[NT][kSteps][2];
    int lo[NT][2], hi[NT][2];  // cached tokens that rows 2c, 2c + 1 of a tile see
    int all_lo = 0, all_hi = p.u.end;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      const bool has = r < p.u.rows;
      int token = 0, head = 0;
      if (has) attn_row_of(a, p, r, token, head);
      const uint16_t* q = a.q.data + token * a.q.token_stride + head * a.q.head_stride;
      if constexpr (B == 4 || B == 6) {  // 8 neighbouring dims are two steps, in the unpackers' order of pairs
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i) {
          const int d = B == 4 ? 32 * i + 8 * c : c * (D / 4) + 8 * i;
          const uint4 v = has ? __ldg(reinterpret_cast<const uint4*>(q + d)) : make_uint4(0, 0, 0, 0);
          bq[nt][2 * i][0] = prmt(v.x, v.z, 0x5410);      // 0, 4
          bq[nt][2 * i][1] = prmt(v.x, v.z, 0x7632);      // 1, 5
          bq[nt][2 * i + 1][0] = prmt(v.y, v.w, 0x5410);  // 2, 6
          bq[nt][2 * i + 1][1] = prmt(v.y, v.w, 0x7632);  // 3, 7
        }
      } else if constexpr (B == 8) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint2 v = has ? __ldg(reinterpret_cast<const uint2*>(q + 16 * i + 4 * c)) : make_uint2(0, 0);
          bq[nt][i][0] = v.x;
          bq[nt][i][1] = v.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          bq[nt][i][0] = has ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * i + 2 * c)) : 0u;
          bq[nt][i][1] = has ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * i + 8 + 2 * c)) : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = p.u.r0 + min(8 * nt + 2 * c + i, p.u.rows - 1), pos = p.u.len - p.u.n + rr / a.group;
        hi[nt][i] = a.causal ? min(pos + 1, p.u.len) : p.u.len;
        lo[nt][i] = a.window > 0 ? pos - a.window + 1 : 0;
        all_lo = max(all_lo, lo[nt][i]);
        all_hi = min(all_hi, hi[nt][i]);
      }
    }
    // bounds of the tokens that all rows see, over the warp
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);

    float o[NT][kSteps][4], l[NT][2];
    float m[NT][2], nbase[NT][2];  // the rows' references, and -m (0 before there is one)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) l[nt][i] = 0.f, m[nt][i] = -INFINITY, nbase[nt][i] = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    bool begun = false;            // every row of the lane has a reference
    bool taken = false;            // values of V that are not finite were taken out

    for (int t = t0; t < t1; ++t, ++tile) {
      const int here = st;
      const uint32_t parity = ph;
      if (++st == C::kStages) {
        st = 0;
        ph ^= 1;
      }
      if (C::kAlternate && (tile & 1) != turn) continue;
      // a wait that gave up leaves the unit as it is, but no barrier below:
      // all warps go through the same ones, whichever of them saw the flag
      if (!mbar_wait_warp(smem_u32(&full[here]), parity, abort_flag, a)) break;
      const uint32_t kbase = smem_u32(smem + here * C::kStage), vbase = kbase + C::kArray, sbase = vbase + C::kArray;
      const int first = t * kTile + row0;
      if (first < end && first + 16 * kSlices > begin) {  // some token of the slices is seen
        // ---------------------------------------------------------- S^T = K Q^T
        float s[kSlices][NT][4];
        {
          float s2[kSlices][NT][4];
#pragma unroll
          for (int h = 0; h < kSlices; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[h][nt][i] = s2[h][nt][i] = 0.f;
#pragma unroll
          for (int h = 0; h < kSlices; ++h) scores<B, D, NT>(kbase, row0 + 16 * h, lane, bq, s[h], s2[h]);
#pragma unroll
          for (int h = 0; h < kSlices; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[h][nt][i] += s2[h][nt][i];
        }
        // ---------------------------------------------------------- softmax
        const bool all_see = first >= all_lo && first + 16 * kSlices <= all_hi;
        float ks[kSlices][2], vs[kSlices][2];
        uint32_t vtop = 0;
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < kSlices; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // the lane's two tokens of a slice
            ks[h][e] = a.scale_log2;
            vs[h][e] = 1.f;
            if constexpr (kQuant) {
              const int tok = row0 + 16 * h + token_at<B>(g + 8 * e);
              ks[h][e] *= attn_key_scale(lds16(sbase + 2 * tok));
              uint32_t v = lds16(sbase + C::kScale + 2 * tok);
              if (t * kTile + tok >= end) v = 0;  // whatever the slots past the end hold
              vtop = max(vtop, v);
              vs[h][e] = half_bits_to_float(v);
            }
          }
        if (kQuant && vtop >= 0x7C00u) {  // one of them is not finite (or below 0, which no codec gives)
#pragma unroll
          for (int h = 0; h < kSlices; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!(fabsf(vs[h][e]) < INFINITY)) ks[h][e] = NAN, vs[h][e] = 0.f;
        }
        // exponents: scores less the rows' references, and the lane's largest
#pragma unroll
        for (int h = 0; h < kSlices; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = first + 16 * h + token_at<B>(g + 8 * e);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float x = fmaf(s[h][nt][2 * e + i], ks[h][e], nbase[nt][i]);
                if (!all_see && (at < lo[nt][i] || at >= hi[nt][i])) x = -INFINITY;
                s[h][nt][2 * e + i] = x;
                top = fmaxf(top, x);
              }
          }
        // ---- references, see attn_lag
        constexpr float kLag = attn_lag<B>();
        const float ve = kQuant ? static_cast<float>(static_cast<int>(vtop >> 10) - 15) : 0.f;
        if (__any_sync(0xffffffffu, !begun || top + ve > kLag)) {
          begun = true;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = -INFINITY;
#pragma unroll
              for (int h = 0; h < kSlices; ++h)
                if constexpr (kQuant)
                  mx = fmaxf(mx, fmaxf(s[h][nt][i] + attn_value_exponent(vs[h][0]),
                                       s[h][nt][i + 2] + attn_value_exponent(vs[h][1])));
                else
                  mx = fmaxf(mx, fmaxf(s[h][nt][i], s[h][nt][i + 2]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              mx -= nbase[nt][i];  // the largest score and exponent
              const float m1 = mx > m[nt][i] + kLag ? mx : m[nt][i];  // m = -inf: mx, where anything is seen
              const float nb1 = m1 == -INFINITY ? 0.f : -m1;
              const float d = nb1 - nbase[nt][i];
              f[i] = m[nt][i] == -INFINITY ? 1.f : exp2_fast(d);  // -inf: o and l are zeros
#pragma unroll
              for (int h = 0; h < kSlices; ++h) s[h][nt][i] += d, s[h][nt][i + 2] += d;
              m[nt][i] = m1;
              nbase[nt][i] = nb1;
              begun &= m1 != -INFINITY;
              l[nt][i] *= f[i];
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              o[nt][i][0] *= f[0], o[nt][i][1] *= f[1];
              o[nt][i][2] *= f[0], o[nt][i][3] *= f[1];
            }
          }
        }
        uint32_t pb[kSlices][NT][2];  // weights times V's scales, as B fragments
#pragma unroll
        for (int h = 0; h < kSlices; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w0 = exp2_fast(s[h][nt][2 * e]), w1 = exp2_fast(s[h][nt][2 * e + 1]);
              l[nt][0] += w0;
              l[nt][1] += w1;
              const __half2 w = __floats2half2_rn(w0 * vs[h][e], w1 * vs[h][e]);
              pb[h][nt][e] = transpose8(*reinterpret_cast<const uint32_t*>(&w));
            }
        // ---------------------------------------------------------- O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < kSlices; ++h) {
          Clean ca, cb;
          if (B == 16 && !all_see) {
            const int x = first + 16 * h + 2 * c;
            ca.two(x, begin, end, all_lo, all_hi);
            cb.two(x + 8, begin, end, all_lo, all_hi);
          }
          values<B, D, NT>(vbase, row0 + 16 * h, lane, !all_see, ca, cb, taken, pb[h], o);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[here]));
    }

    // -------------------------------------------------------------- the warps' results to one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], d);
        if (g == 0) {
          stat_m[warp * C::kRows + 8 * nt + 2 * c + i] = l[nt][i] != 0.f ? -nbase[nt][i] : -INFINITY;
          stat_l[warp * C::kRows + 8 * nt + 2 * c + i] = l[nt][i];
        }
      }
    if constexpr (!kQuant) {
      taken = __any_sync(0xffffffffu, taken);
      if (lane == 0) cleaned[warp] = taken;
    }
    consumer_sync();
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) mm = fmaxf(mm, stat_m[w * C::kRows + 8 * nt + 2 * c + i]);
        f[nt][i] = l[nt][i] != 0.f ? exp2_fast(-nbase[nt][i] - mm) : 0.f;
      }
    const auto put = [&](float* region, bool add) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float y = o[nt][i][2 * h + j] * f[nt][j];
              float* at = region + (8 * nt + 2 * c + j) * D + dim_of<B, D>(i, h, g);
              *at = add ? *at + y : y;
            }
    };
    if constexpr (C::kRegions > 1) {
      put(merge + warp * C::kRows * D, false);
      consumer_sync();
    } else {
      for (int w = 0; w < kConsumers; ++w) {
        if (w == warp) put(merge, w > 0);
        consumer_sync();
      }
    }
    // 128 threads: 4 dims of a row each
    const int c0 = p.whole ? 0 : attn_cta_of(state.s, p.first), c1 = p.whole ? 0 : attn_cta_of(state.s, p.first + p.u.tiles - 1);
    const int me = blockIdx.x;
    float* slot = p.whole ? nullptr : attn_slot(a, me, me == c0, C::kFloats);
    for (int e = threadIdx.x; e < p.u.rows * (D / 4); e += kConsumers * 32) {
      const int r = e / (D / 4), col = e % (D / 4);
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) mm = fmaxf(mm, stat_m[w * C::kRows + r]);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float lw = stat_l[w * C::kRows + r];
        if (lw != 0.f) ll += lw * exp2_fast(stat_m[w * C::kRows + r] - mm);
      }
      float4 y = *reinterpret_cast<const float4*>(merge + r * D + 4 * col);
#pragma unroll
      for (int w = 1; w < C::kRegions; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(merge + (w * C::kRows + r) * D + 4 * col);
        y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
      }
      if (p.whole) {
        int token, head;
        attn_row_of(a, p, r, token, head);
        const float inv = ll != 0.f ? 1.f / ll : 0.f;
        uint2 out;
        out.x = float_to_half_bits(y.x * inv) | (float_to_half_bits(y.y * inv) << 16);
        out.y = float_to_half_bits(y.z * inv) | (float_to_half_bits(y.w * inv) << 16);
        *reinterpret_cast<uint2*>(a.out.data + token * a.out.token_stride + head * a.out.head_stride + 4 * col) = out;
        if (col == 0) attn_store_lse(a, token, head, mm, ll);
      } else {
        *reinterpret_cast<float4*>(slot + r * D + 4 * col) = y;
        if (col == 0) slot[C::kRows * D + r] = mm, slot[C::kRows * D + C::kRows + r] = ll;
      }
    }
    if (!kQuant && (cleaned[0] | cleaned[1] | cleaned[2] | cleaned[3])) {
      __syncwarp();  // the stores above come first, whatever their types
      for (int e = threadIdx.x; e < p.u.rows * (D / 4); e += kConsumers * 32) {  // each its own stores
        const int r = e / (D / 4), d = 4 * (e % (D / 4));
        int token, head;
        attn_row_of(a, p, r, token, head);
        attn_put_back<D>(a, p, kTile, r, d, a.out.data + token * a.out.token_stride + head * a.out.head_stride,
                         p.whole ? nullptr : slot + r * D);
      }
    }
    if (!p.whole) {
      __threadfence();
      consumer_sync();
      if (threadIdx.x == 0) {
        const int last = atomicAdd(a.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
        if (last) a.counters[c0] = 0u;
        *is_last = last;
      }
      consumer_sync();
      if (*is_last) {
        __threadfence();
        attn_join<C::kRows, D>(a, p, c0, c1, threadIdx.x, kConsumers * 32);
      }
    }
    consumer_sync();  // merge and the statistics are free again
  }
}

// ---------------------------------------------------------------- host

inline bool encode_cache(CUtensorMap* map, const void* base, const exq_kv_cache& c, int part_words,
                         CUtensorMapSwizzle swizzle) {
  EncodeTiled enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t words = static_cast<cuuint64_t>(c.D) * c.bits / 32;
  const cuuint64_t dims[3] = {words, static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.n_pages) * c.n_kv_heads};
  const cuuint64_t strides[2] = {words * 4, words * 4 * c.page_size};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(part_words), static_cast<cuuint32_t>(std::min(kTile, c.page_size)), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int B, int D, int NT>
exq_status launch(const AttnCall& call, const AttnArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<B, D, NT>;
  Maps maps;
  constexpr CUtensorMapSwizzle kSwizzle = B == 6                ? CU_TENSOR_MAP_SWIZZLE_NONE
                                          : C::kPartBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                          : C::kPartBytes == 64  ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                 : CU_TENSOR_MAP_SWIZZLE_32B;
  if (!encode_cache(&maps.k, a.codes[0], *call.cache, C::kPartBytes / 4, kSwizzle) ||
      !encode_cache(&maps.v, a.codes[1], *call.cache, C::kPartBytes / 4, kSwizzle))
    return EXQ_ERR_CUDA;
  auto fn = attn_split_kernel<B, D, NT>;
  static PerDevice state;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || !state.once(dev, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) == cudaSuccess;
      }))
    return EXQ_ERR_CUDA;
  // Units cut into more than 32 pieces take two CTAs an SM: fewer pieces to
  // join. us with two and with all, D = 128 (three): 8 units of 131072 tokens Q8
  // 62 / 66, Q4 48.5 / 49.4, of 16384 Q4 20 / 26; past the limit 16 units of up
  // to 131072 Q4 66 / 64, Q8 88 / 90, 32 units of 32768 Q4 43.6 / 40.3. D = 64
  // (four), Q4: 4 units of 131072 37 / 51, 12 40 / 43, 16 53 / 49 (of 16384 18 /
  // 25); past the limit 24 of 65536 32 / 33.
  const long long units = static_cast<long long>(a.n_seqs) * a.row_blocks * a.n_kv_heads;
  const int ctas = units * 32 < static_cast<long long>(sms) * C::kCtas ? std::min(C::kCtas, 2) : C::kCtas;
  fn<<<std::min(sms * ctas, kAttnMaxCtas), kThreads, C::kSmem, stream>>>(maps, a);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

template <int B>
exq_status launch_bits(const AttnCall& call, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream) {
  const bool one = unit_rows == 8;
  switch (call.cache->D) {
    case 64: return one ? launch<B, 64, 1>(call, a, sms, stream) : launch<B, 64, 2>(call, a, sms, stream);
    case 128: return one ? launch<B, 128, 1>(call, a, sms, stream) : launch<B, 128, 2>(call, a, sms, stream);
    default: return launch<B, 256, 1>(call, a, sms, stream);
  }
}

// unit_rows for sequences of `rows` rows
inline int rows_of(int D, long long rows) { return D == 256 || rows <= 8 ? 8 : 16; }

}  // namespace split

exq_status launch_attn_split4(const AttnCall& c, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream);
exq_status launch_attn_split6(const AttnCall& c, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream);
exq_status launch_attn_split8(const AttnCall& c, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream);
exq_status launch_attn_split16(const AttnCall& c, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream);

}  // namespace exq
