// Attention of many rows over the paged cache (chunks of prompts) on the
// 5th-generation tensor cores: S = Q K^T and O += P V with fp32 sums in tensor
// memory. The multiplications are the bound.
//
// A unit is 256 rows (128 for D = 256) of one KV head: two M = 128 tiles, each
// with its own O and two S buffers of 64 cached tokens in tensor memory, all
// 512 columns of it for D = 128. The scores of the next tile are computed
// while a tile's softmax runs, so the softmax never waits for the round trip
// through the tensor cores (with one S of 128 tokens, its 2000 cycles and the
// round trip's 2300 came one after the other). Roles of a CTA, one per SM:
//
//   warps 0-7   softmax: S once into registers; the weights go back as fp16
//               over S, the A operand of P V; the sums of weights; the
//               epilogue. A row's reference is raised, and O rescaled, only
//               when a score exceeds it by more than attn_lag. So most tiles
//               need no row maximum over lanes, one vote does.
//   warps 8-11  dequantisers: packed tiles in shared memory become the
//               integers (u - z), exact in fp16, in the MMA's 128-byte
//               swizzle, once for all rows of the unit. The groups' scales
//               stay in fp32 beside the tile and multiply S's columns (K) and
//               the weights (V) in the softmax: rounding (u - z) s to fp16
//               here instead would be one rounding more per cached value. For
//               fp16 pages, which TMA brings in place, they only clean V's
//               tokens that not every row sees. They also bring Q.
//   warp 12     issues S = Q K^T, warps 14 and 15 O += P V of the two M tiles.
//               An MMA is accepted about when the one before is done, so a
//               warp's wait on a barrier (100 to 300 cycles beside busy warps,
//               even if it is complete) leaves the tensor cores idle; with
//               three issuers another's MMAs fill the gap (one issuer: 2500
//               cycles a tile, of which 1260 were MMAs).
//   warp 13     issues the TMA copies.
//
// K is K-major (tokens x 64 dims per 128-byte swizzled row); V has the same
// layout and is the MN-major B operand, so nothing is transposed.
//
// 2048 tokens over 16000 (8 KV heads of 128, 8 query heads each, Q4): 882 us,
// 1139 TFLOPS, 60 % of a large library product's rate; prompts up to 3500
// tokens in a window of 1024 (fp16): 230 us. Neither the tensor pipe (33 and
// 13 % of the time) nor the issue slots are full: the waits of the chain from
// scores to weights to P V, and of a unit's beginning and end, are the time.
#pragma once

#include <algorithm>
#include <type_traits>

#include "exq_attn_split.cuh"

namespace exq {
namespace chunk {

constexpr int kSoftmaxThreads = 256;
constexpr int kDequantThreads = 128;
constexpr int kThreads = 512;  // registers move between whole groups of 4 warps
constexpr int kScoreWarp = 12, kTmaWarp = 13, kValueWarp = 14;
constexpr int kTile = split::kTile;

// Registers a thread: the block is launched with kLaunchRegs and hands those
// of the MMA's group to the softmax. The shares may not add up to more than
// the launch's, or an increase would never be granted.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 152, kDequantRegs = 112, kIssueRegs = 96;
static_assert(2 * kSoftmaxRegs + kDequantRegs + kIssueRegs <= 4 * kLaunchRegs, "register shares");

template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int B, int D>
struct Cfg {
  using Packed = split::Cfg<B, D, 1>;                // the packed tile's layout, as TMA writes it
  static constexpr int kStreams = D == 256 ? 1 : 2;  // M = 128 tiles of a unit
  static constexpr int kRows = 128 * kStreams;
  static constexpr int kSlabs = D / 64;              // 64 dims: one 128-byte swizzled row
  static constexpr int kArray = kTile * D * 2;       // K or V of a stage, fp16
  static constexpr int kStages = D == 256 ? 2 : B == 16 ? 4 : 3;  // of K and V together
  static constexpr int kOffV = 0;
  static constexpr int kOffK = kStages * kArray;
  static constexpr int kOffQ = 2 * kStages * kArray;
  static constexpr int kOffPacked = kOffQ + kRows * D * 2;
  // a packed stage is one tile of K or of V with its scales
  static constexpr int kPacked = B == 16 ? 0 : (Packed::kArray + Packed::kScale + 1023) / 1024 * 1024;
  static constexpr int kRoom = 227 * 1024 - 1024 - kOffPacked - 4 * 3 * kTile * 4 - 64 - kStreams * 4 * 2048 -
                               kThreads / 32 * static_cast<int>(sizeof(AttnState)) - 512;
  static constexpr int kPackedFit = B == 16 ? 0 : kRoom / kPacked;
  static constexpr int kPackedStages = kPackedFit > 8 ? 8 : kPackedFit;
  static constexpr int kOffScale = kOffPacked + kPackedStages * kPacked;  // [4][sk, sv][kTile] fp32, [4][kTile] sv's exponents
  static constexpr int kOffExps = kOffScale + 4 * 3 * kTile * 4;          // [4][2]: V's largest exponents
  static constexpr int kOffStage = kOffExps + 64;                         // 32 rows of 64 bytes a softmax warp
  static constexpr int kOffState = kOffStage + kStreams * 4 * 2048;       // a warp's place each
  static constexpr int kOffBar = kOffState + kThreads / 32 * static_cast<int>(sizeof(AttnState));
  static constexpr int kSmem = 1024 + kOffBar + 512;
  static constexpr int kFloats = kRows * (D + 2);
  static_assert(B == 16 || kPackedStages >= 1, "a packed stage");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // tensor memory columns
  static constexpr int kTmemS = 0;                   // [stream][2][kTile]
  static constexpr int kTmemO = 256;                 // [stream][D]
};

using split::Maps;

struct Extra {
  float scale;       // |scale| log2(e); 0 is passed as 2^-126
  int negate;        // scale < 0: the MMA negates Q
};

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The MMA warp issues as a whole, one lane elected in each instruction: the
// operands then stay in uniform registers. Issued from a branch that only
// lane 0 takes, an M = 128, N = 128, K = 16 product took 90 to 140 cycles
// beside busy softmax warps; this way 64, the tensor cores' own time.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
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
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
using split::uniform;
// Copies that the lane of a box issues on its own. Issued by the whole warp
// (as in the packed-code kernel) this kernel took 20 % longer on quantised
// pages: the copies have time here, and the warp's issue slots have not.
__device__ __forceinline__ void lane_tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void lane_bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
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
// 16 lanes x 64 columns as the fragments of mma.sync: register 4 j + 2 i + k is
// row lane / 4 + 8 i, column 8 j + 2 (lane % 4) + k
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// and 16 lanes x 16 columns, loaded, scaled by the rows' factors and stored back
__device__ __forceinline__ void tmem_scale16(uint32_t taddr, float f0, float f1) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * ((i >> 1) & 1 ? f1 : f0));
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 lanes x 32 columns of fp16 pairs: register 2 j + i is row lane / 4 + 8 i, column 4 j + lane % 4
__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// both halves of a warp's 32 rows
__device__ __forceinline__ void tmem_wait_frag(uint32_t (&r)[2][32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0][0]), "+r"(r[0][1]), "+r"(r[0][2]), "+r"(r[0][3]), "+r"(r[0][4]), "+r"(r[0][5]),
                 "+r"(r[0][6]), "+r"(r[0][7]), "+r"(r[0][8]), "+r"(r[0][9]), "+r"(r[0][10]), "+r"(r[0][11]),
                 "+r"(r[0][12]), "+r"(r[0][13]), "+r"(r[0][14]), "+r"(r[0][15]), "+r"(r[0][16]), "+r"(r[0][17]),
                 "+r"(r[0][18]), "+r"(r[0][19]), "+r"(r[0][20]), "+r"(r[0][21]), "+r"(r[0][22]), "+r"(r[0][23]),
                 "+r"(r[0][24]), "+r"(r[0][25]), "+r"(r[0][26]), "+r"(r[0][27]), "+r"(r[0][28]), "+r"(r[0][29]),
                 "+r"(r[0][30]), "+r"(r[0][31])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[1][0]), "+r"(r[1][1]), "+r"(r[1][2]), "+r"(r[1][3]), "+r"(r[1][4]), "+r"(r[1][5]),
                 "+r"(r[1][6]), "+r"(r[1][7]), "+r"(r[1][8]), "+r"(r[1][9]), "+r"(r[1][10]), "+r"(r[1][11]),
                 "+r"(r[1][12]), "+r"(r[1][13]), "+r"(r[1][14]), "+r"(r[1][15]), "+r"(r[1][16]), "+r"(r[1][17]),
                 "+r"(r[1][18]), "+r"(r[1][19]), "+r"(r[1][20]), "+r"(r[1][21]), "+r"(r[1][22]), "+r"(r[1][23]),
                 "+r"(r[1][24]), "+r"(r[1][25]), "+r"(r[1][26]), "+r"(r[1][27]), "+r"(r[1][28]), "+r"(r[1][29]),
                 "+r"(r[1][30]), "+r"(r[1][31])
               :
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

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}

// byte offset of the 16-byte chunk of dims [8 ch, 8 ch + 8) of row `row` in an
// operand of `rows` rows: 64-dim slabs of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t operand_at(int rows, int row, int ch) {
  return (ch >> 3) * (rows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); }

// ---- dequantisers: an item is the codes of one 12- (Q6) or 16-byte piece of
// a token's row; consecutive threads hold 8 tokens of one piece, so that the
// loads (TMA's swizzle) and the 16-byte stores (the MMA's) fall on different
// banks
template <int B, int D>
struct Item {
  static constexpr int kWords = B == 6 ? 3 : 4;
  static constexpr int kCodes = kWords * 32 / B;            // 32 or 16
  static constexpr int kPerRow = D / kCodes;
  static constexpr int kItems = kTile * kPerRow / kDequantThreads;
};

// Each 8 codes become a 16-byte chunk of (u - z): Q8 in the dims' order, Q4
// and Q6 as the unpackers' pairs (0 4 1 5 2 6 3 7), the order in which Q is
// loaded and O stored
template <int B, int D>
__device__ __forceinline__ void dequant(uint32_t src, uint32_t dst, int tid) {
  using I = Item<B, D>;
  using P = typename Cfg<B, D>::Packed;
#pragma unroll
  for (int it = 0; it < I::kItems; ++it) {
    const int i = it * kDequantThreads + tid;
    const int row = (i & 7) + 8 * (i / (8 * I::kPerRow)), piece = (i >> 3) % I::kPerRow;
    uint32_t w[4];
    if constexpr (B == 6) {
#pragma unroll
      for (int j = 0; j < 3; ++j) w[j] = split::lds32(src + row * P::kRowBytes + piece * 12 + 4 * j);
    } else {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(src + split::chunk_at<P>(row, piece)));
    }
    const int ch = piece * (I::kCodes / 8);
#pragma unroll
    for (int j = 0; j < I::kCodes / 8; ++j) {
      uint32_t v[4];
      if constexpr (B == 4) {
        unpack8<4>(w[j], 0u, v);
      } else if constexpr (B == 8) {
        v[0] = split::q8_pair(w[2 * j], 0x4140), v[1] = split::q8_pair(w[2 * j], 0x4342);
        v[2] = split::q8_pair(w[2 * j + 1], 0x4140), v[3] = split::q8_pair(w[2 * j + 1], 0x4342);
      } else {
        if (j == 0) unpack8<6>(w[0], w[1], v);
        else unpack8<6>(fshr(w[1], w[2], 16), w[2] >> 16, v);
      }
      sts128(dst + operand_at(kTile, row, ch + j), v[0], v[1], v[2], v[3]);
    }
  }
}

// A position in a ring of N stages and the parity of its pass.
template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1;
    }
  }
};

// attn_put_back for a whole row of a unit. Rare, so a call of its own.
template <int D, int FLOATS>
__device__ __noinline__ void put_back_row(const AttnArgs& a, const AttnPiece& p, int row, bool begins) {
  int tk, hd;
  attn_row_of(a, p, row, tk, hd);
#pragma unroll 1
  for (int d = 0; d < D; d += 4)
    attn_put_back<D>(a, p, kTile, row, d, a.out.data + tk * a.out.token_stride + hd * a.out.head_stride,
                     p.whole ? nullptr : attn_slot(a, blockIdx.x, begins, FLOATS) + row * D);
}

template <int B, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, const __grid_constant__ Extra x) {
  using C = Cfg<B, D>;
  using P = typename C::Packed;
  constexpr bool kQuant = B != 16;
  constexpr bool kPairs = B == 4 || B == 6;  // dims in the unpackers' order
  constexpr int T = kTile;
  constexpr int kNP = kQuant ? C::kPackedStages : 1;
  constexpr int kNS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + C::kOffScale);
  int* exps = reinterpret_cast<int*>(smem + C::kOffExps);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  // Barriers. Tiles are counted over the CTA's whole share; S and P V of tile
  // i complete phase i / 4 of barrier i % 4 of their kinds. P V says too that
  // the stage of K and V and the weights (S's buffer) have been read.
  const uint32_t bar0 = smem_u32(bars);
  const auto s_full = [bar0](uint32_t tile) { return bar0 + 8 * (tile & 3); };
  const auto pv_done = [bar0](uint32_t tile) { return bar0 + 32 + 8 * (tile & 3); };
  const auto w_full = [bar0](int stream, int buf) { return bar0 + 64 + 8 * (2 * stream + buf); };  // weights are there
  const auto kv_full = [bar0](int st) { return bar0 + 96 + 8 * st; };
  const auto packed_full = [bar0](int st) { return bar0 + 128 + 8 * st; };
  const auto packed_empty = [bar0](int st) { return bar0 + 192 + 8 * st; };
  const auto v_ready = [bar0](uint32_t tile) { return bar0 + 256 + 8 * (tile & 3); };  // fp16 pages: V is clean
  const uint32_t q_full = bar0 + 288, drain = bar0 + 296 /* of warps 12, 14, 15 */;
  const auto phase4 = [](uint32_t tile) { return (tile >> 2) & 1; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* is_last = reinterpret_cast<int*>(tmem_slot + 2);
  // The last pieces' numbers (from 1) whose V was cleaned. The dequantisers may
  // be three pieces ahead of the epilogue: the scores of two tiles and their
  // queries are.
  volatile int* cleaned = reinterpret_cast<volatile int*>(tmem_slot + 3);  // [4]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(pv_done(i), C::kStreams);
      mbar_init(w_full(i >> 1, i & 1), 128);
      mbar_init(kv_full(i), kQuant ? kDequantThreads : 1);
      mbar_init(v_ready(i), kDequantThreads);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(packed_full(i), 1);
      mbar_init(packed_empty(i), kDequantThreads);
    }
    mbar_init(q_full, kDequantThreads);
    for (int i = 0; i < 3; ++i) mbar_init(drain + 8 * i, 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) cleaned[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  AttnState& state = reinterpret_cast<AttnState*>(smem + C::kOffState)[warp];
  if (!attn_begin<C::kRows, T>(a, state)) return;  // the whole CTA
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  const AttnPiece& p = state.p;

  if (warp >= kScoreWarp) {
    fewer_regs<kIssueRegs>();
    if (warp == kScoreWarp) {
      // ------------------------------------------------------------ S = Q K^T
      const uint32_t idesc = uniform(instr_desc(T, false, x.negate != 0));
      const uint32_t tm = uniform(tmem + C::kTmemS), sb = uniform(sbase);
      Ring<kNS> r;
      uint32_t g = 0, q_ph = 0;
      bool ok = true;
      while (ok && attn_next<C::kRows, T>(a, state)) {
        const int n = uniform(p.t1 - p.t0), ns = uniform(p.u.rows) > 128 ? C::kStreams : 1;
        ok = mbar_wait_warp(q_full, q_ph, abort_flag, a);
        q_ph ^= 1;
        for (int j = 0; j < n && ok; ++j, ++g) {
          ok = mbar_wait_warp(kv_full(r.st), r.ph, abort_flag, a);
          if (ok && g >= 2) ok = mbar_wait_warp(pv_done(g - 2), phase4(g - 2), abort_flag, a);  // the buffer's last weights
          if (!ok) break;
          tc_after();
          const uint64_t kd = smem_desc(sb + C::kOffK + uniform(r.st) * C::kArray, 16);
          const uint32_t ts = tm + uniform(g & 1) * T;
#pragma unroll
          for (int s = 0; s < C::kStreams; ++s) {
            if (s >= ns) break;
            const uint64_t qd = smem_desc(sb + C::kOffQ + s * (128 * D * 2), 16);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              mma_ss(ts + s * 2 * T, qd + ((i >> 2) * (128 * 128) + (i & 3) * 32) / 16,
                     kd + ((i >> 2) * (T * 128) + (i & 3) * 32) / 16, idesc, i > 0);
          }
          tc_commit(s_full(g));
          r.next();
        }
      }
      tc_commit(drain);
    } else if (warp >= kValueWarp && warp - kValueWarp < C::kStreams) {
      // ------------------------------------------------------------ O += P V of one M tile
      const uint32_t s = uniform(warp - kValueWarp), idesc = uniform(instr_desc(D, true, false));
      const uint32_t to = uniform(tmem + C::kTmemO + s * D), tp = uniform(tmem + C::kTmemS + 2 * s * T), sb = uniform(sbase);
      Ring<kNS> r;
      uint32_t g = 0, w_ph = 0;
      bool ok = true;
      while (ok && attn_next<C::kRows, T>(a, state)) {
        const int n = uniform(p.t1 - p.t0);
        const bool active = uniform(p.u.rows) > 128 * s;
        for (int j = 0; j < n && ok; ++j, ++g, r.next()) {
          const uint32_t buf = uniform(g & 1);
          if (!kQuant && active) ok = mbar_wait_warp(v_ready(g), phase4(g), abort_flag, a);
          ok = ok && mbar_wait_warp(w_full(s, buf), (w_ph >> buf) & 1, abort_flag, a);
          w_ph ^= 1u << buf;
          if (!ok) break;
          if (!active) {  // no rows: keeps the phases whole, and its softmax warps in step
            if (lane == 0) mbar_arrive(pv_done(g));
            continue;
          }
          tc_after();
          const uint64_t vd = smem_desc(sb + C::kOffV + uniform(r.st) * C::kArray, T * 128);
#pragma unroll
          for (int i = 0; i < T / 16; ++i) mma_ts(to, tp + buf * T + 8 * i, vd + i * 128, idesc, i > 0 ? 1 : j > 0);
          tc_commit(pv_done(g));
        }
      }
      tc_commit(drain + 8 * (1 + s));
    } else if (warp == kTmaWarp && a.starve == 0) {  // test hook: the other roles' waits run out
      // ------------------------------------------------------------ TMA producer
      const int box = min(T, a.page_size), boxes = T / box;  // tokens of a box, boxes of a tile
      Ring<kNP> pr;
      Ring<kNS> r;
      uint32_t g = 0;          // tiles
      long long issued = 0;    // stages filled
      bool ok = true;
      while (ok && attn_next<C::kRows, T>(a, state)) {
        const int32_t* table = a.page_table + static_cast<long long>(p.u.b) * a.max_pages;
        const int t0 = p.t0, t1 = p.t1, head = p.head, begin = p.u.begin, end = p.u.end;
        const int b0 = t0 * boxes, b1 = t1 * boxes;
        const auto page_of = [&](int bx) {  // -1: nothing to copy
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
        for (int t = t0; t < t1; ++t, ++g) {
          if (t * boxes >= have + 32) {
            have += 32;
            page = next;
            next = page_of(have + 32 + lane);
          }
          const int mine = __shfl_sync(0xffffffffu, page, (t * boxes - have + (lane & (boxes - 1))) & 31);
          const bool copy = lane < boxes && mine >= 0;
          const unsigned n = __popc(__ballot_sync(0xffffffffu, copy));
          const int slot = (t * T + lane * box) & (a.page_size - 1), block = mine * a.n_kv_heads + head;
          if constexpr (kQuant) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              ok = ok && mbar_wait_warp(packed_empty(pr.st), pr.ph ^ 1, abort_flag, a);
              if (!ok) break;
              const uint32_t full = packed_full(pr.st), base = sbase + C::kOffPacked + pr.st * C::kPacked;
              if (lane == 0) mbar_expect_tx(full, n * box * (P::kRowBytes + 2));
              __syncwarp();
              if (copy) {
#pragma unroll
                for (int i = 0; i < P::kParts; ++i)
                  lane_tma_load_3d(base + i * (T * P::kPartBytes) + lane * box * P::kPartBytes, which ? &maps.v : &maps.k,
                                     i * (P::kPartBytes / 4), slot, block, full);
                lane_bulk_load(base + P::kArray + lane * box * 2,
                                 a.scales[which] + static_cast<long long>(block) * a.page_size + slot, box * 2, full);
              }
              pr.next();
              ++issued;
            }
            if (!ok) break;
          } else {
            if (g >= kNS) ok = mbar_wait_warp(pv_done(g - kNS), phase4(g - kNS), abort_flag, a);
            if (!ok) break;
            const uint32_t full = kv_full(r.st);
            if (lane == 0) mbar_expect_tx(full, n * box * D * 4);
            __syncwarp();
            if (copy) {
              const uint32_t at = sbase + r.st * C::kArray + lane * box * 128;
#pragma unroll
              for (int i = 0; i < C::kSlabs; ++i) {
                lane_tma_load_3d(at + C::kOffK + i * (T * 128), &maps.k, i * 32, slot, block, full);
                lane_tma_load_3d(at + C::kOffV + i * (T * 128), &maps.v, i * 32, slot, block, full);
              }
            }
            r.next();
            ++issued;
          }
        }
      }
      // every copy lands before the CTA may go
      constexpr int kRing = kQuant ? kNP : kNS;
      for (long long i = max(0ll, issued - kRing); i < issued; ++i) {
        const int st = static_cast<int>(i % kRing);
        for (int k = 0; k < a.wait_limit; ++k)
          if (mbar_try_wait(kQuant ? packed_full(st) : kv_full(st), (i / kRing) & 1)) break;
      }
    }
  } else if (warp >= kSoftmaxThreads / 32) {
    // -------------------------------------------------------------- dequantisers
    fewer_regs<kDequantRegs>();
    const int tid = threadIdx.x - kSoftmaxThreads;
    Ring<kNP> pr;
    Ring<kNS> r;
    uint32_t g = 0;  // tiles
    bool ok = true;
    while (ok && attn_next<C::kRows, T>(a, state)) {
      // ---- Q: [M tile][slab][128 rows][128 bytes]; rows past the unit are
      // zeros. The last S of the unit before has been computed.
      if (g > 0) ok = mbar_wait_warp(s_full(g - 1), phase4(g - 1), abort_flag, a);
      if (!ok) break;
      const int rows = p.u.rows, q_rows = rows > 128 ? C::kRows : 128;
      {
        // A thread's chunk of the dims (for D = 256 also the one 16 on) and
        // its first row; its rows step by kStep. Eight threads hold
        // neighbouring rows of one chunk, so that their stores fall on
        // different banks; 8 loads at a time.
        constexpr int kPer = D == 256 ? 2 : 1, kStep = D == 64 ? 16 : 8, kBatch = 8 / kPer;
        const int ch = (tid >> 3) & (D == 64 ? 7 : 15);
        int row = (tid & 7) + (D == 64 ? 8 * (tid >> 6) : 0);
        const int group = a.group, down = kStep / group, over = kStep - down * group;
        const long long ts = a.q.token_stride, hs = a.q.head_stride;
        int head = (p.u.r0 + row) % group;
        const uint16_t* src = a.q.data + (p.u.q0 + (p.u.r0 + row) / group) * ts + (p.head * group + head) * hs + 8 * ch;
        const long long step = down * ts + over * hs, wrap = ts - group * hs;  // and from the last head to the next token
        for (int i0 = 0; i0 < q_rows; i0 += kBatch * kStep) {
          uint4 v[kBatch][kPer];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
              v[j][k] = row + j * kStep < rows ? __ldg(reinterpret_cast<const uint4*>(src + 128 * k)) : make_uint4(0, 0, 0, 0);
            src += step;
            head += over;
            if (head >= group) {
              head -= group;
              src += wrap;
            }
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int r = row + j * kStep;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              uint4 u = v[j][k];
              if constexpr (kPairs)
                u = make_uint4(prmt(u.x, u.z, 0x5410), prmt(u.x, u.z, 0x7632), prmt(u.y, u.w, 0x5410), prmt(u.y, u.w, 0x7632));
              sts128(sbase + C::kOffQ + (r >> 7) * (128 * D * 2) + operand_at(128, r & 127, ch + 16 * k), u.x, u.y, u.z, u.w);
            }
          }
          row += kBatch * kStep;
        }
      }
      async_fence();
      mbar_arrive(q_full);

      const int t1 = p.t1, end = p.u.end;
      AttnSpan all;
      if constexpr (!kQuant) all = attn_seen_by_all(a, p.u);
      for (int t = p.t0; t < t1 && ok; ++t, ++g) {
        if constexpr (kQuant) {
          if (g >= kNS) ok = mbar_wait_warp(pv_done(g - kNS), phase4(g - kNS), abort_flag, a);
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            ok = ok && mbar_wait_warp(packed_full(pr.st), pr.ph, abort_flag, a);
            if (!ok) break;
            const uint32_t src = sbase + C::kOffPacked + pr.st * C::kPacked;
            uint32_t bits = tid < T ? split::lds16(src + P::kArray + 2 * tid) : 0;  // ahead of its use
            dequant<B, D>(src, sbase + (which ? C::kOffV : C::kOffK) + r.st * C::kArray, tid);
            // scales, zero past the end. Four tiles' are kept, and P V of the
            // tile kNS <= 3 ago, so every weight of the one four ago, is done
            if (tid < T) {
              if (tid >= end - t * T) bits = 0;
              scales[(2 * (g & 3) + which) * T + tid] = which ? half_bits_to_float(bits) : attn_key_scale(bits) * x.scale;
              if (which) {
                const int e = static_cast<int>(__reduce_max_sync(0xffffffffu, bits) >> 10) & 31;
                if (lane == 0) exps[2 * (g & 3) + (tid >> 5)] = e;
                // once here: computed in the softmax, code that a unit runs once or
                // twice, a prompt of 2048 tokens took 149 us for 142 (Q4)
                scales[(8 + (g & 3)) * T + tid] = attn_value_exponent(half_bits_to_float(bits));
                if (!attn_finite(bits)) {
                  scales[2 * (g & 3) * T + tid] = NAN;
                  scales[(2 * (g & 3) + 1) * T + tid] = 0.f;
                }
              }
            }
            mbar_arrive(packed_empty(pr.st));
            pr.next();
          }
          if (!ok) break;
          async_fence();
          mbar_arrive(kv_full(r.st));
        } else {
          ok = mbar_wait_warp(kv_full(r.st), r.ph, abort_flag, a);
          if (!ok) break;
          if (t * T < all.lo || (t + 1) * T > all.hi) {  // tokens that not every row sees
            // A thread has one or two 16-byte chunks of every kStep-th row.
            // Tiles whose tokens are all seen by some row are looked over
            // first (x 0 + 0 is NaN where x is not finite): most are clean.
            constexpr int kPer = D == 64 ? 8 : 16, kStep = kDequantThreads / kPer, kParts = D / 8 / kPer;
            const int row0 = tid / kPer;
            const uint32_t own = sbase + C::kOffV + r.st * C::kArray + operand_at(T, row0, tid % kPer);
            uint32_t sum = 0;
            const int begin = p.u.begin;
            const bool all_there = t * T >= begin && (t + 1) * T <= end;
            if (all_there) {
#pragma unroll
              for (int i = 0; i < T / kStep * kParts; ++i) {
                uint32_t v[4];
                lds128(own + (i % kParts) * (2 * T * 128) + i / kParts * (kStep * 128), v);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = hfma2(v[j], 0u, sum);
              }
            }
            if (!all_there || sum != 0) {
#pragma unroll 1
              for (int i = 0; i < T / kStep * kParts; ++i) {
                const int at = t * T + row0 + i / kParts * kStep;
                if (at >= all.lo && at < all.hi) continue;
                const uint32_t to = own + (i % kParts) * (2 * T * 128) + i / kParts * (kStep * 128);
                uint32_t v[4] = {0, 0, 0, 0}, out = 1;
                if (at >= begin && at < end) {
                  lds128(to, v);
                  out = 0;
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const uint32_t m = attn_not_finite(v[j], 0x80008000u);
                    v[j] &= ~m;
                    out |= m;
                  }
                  if (out) cleaned[state.number & 3] = state.number;
                }
                if (out) sts128(to, v[0], v[1], v[2], v[3]);
              }
              async_fence();
            }
          }
          mbar_arrive(v_ready(g));
        }
        r.next();
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    more_regs<kSoftmaxRegs>();
    // A warp has 32 rows (its lanes of tensor memory). S is read as fragments:
    // a thread holds 4 rows (k: 8 k + lane / 4) and, of each 8 columns, two, so
    // that a pair of scales out of shared memory serves 4 rows.
    const int s = C::kStreams == 2 ? warp >> 2 : 0;
    const bool works = C::kStreams == 2 || warp < 4;
    const int row0 = s * 128 + (warp & 3) * 32;           // the warp's first row of the unit
    const int row = row0 + lane;                          // the epilogue's
    const int col2 = 2 * (lane & 3);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    constexpr uint32_t kHalf = 16u << 16;                 // 16 lanes on
    const uint32_t t_o = tmem + lane_base + C::kTmemO + s * D;
    uint32_t g = 0;                                       // tiles
    bool ok = true;
    while (attn_next<C::kRows, T>(a, state)) {
      const bool active = works && s * 128 < p.u.rows;    // warp-uniform, the same for the stream's warps
      float m[4], nbase[4];                               // references, and -m (0 before there is one)
      uint64_t sum[4];                                    // of weights, even and odd columns
      int lo[4], hi[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = -INFINITY, nbase[k] = 0.f, sum[k] = 0;
      if (active) {
        int all_lo = 0, all_hi = p.u.end;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = p.u.r0 + min(row0 + 8 * k + (lane >> 2), p.u.rows - 1), pos = p.u.len - p.u.n + rr / a.group;
          hi[k] = a.causal ? min(pos + 1, p.u.len) : p.u.len;
          lo[k] = a.window > 0 ? pos - a.window + 1 : 0;
          all_lo = max(all_lo, lo[k]);
          all_hi = min(all_hi, hi[k]);
        }
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);
        bool begun = false;  // every row of the thread has a reference
        const int t0 = p.t0, t1 = p.t1;
        for (int t = t0; t < t1 && ok; ++t, ++g) {
          ok = mbar_wait_warp(s_full(g), phase4(g), abort_flag, a);
          if (!ok) break;
          tc_after();
          const int buf = g & 1;
          const uint32_t t_s = tmem + lane_base + C::kTmemS + (2 * s + buf) * T;
          const float* sk = scales + 2 * (g & 3) * T + col2;
          const float* sv = sk + T;
          uint32_t r[2][32];
          tmem_ld_frag(t_s, r[0]);
          tmem_ld_frag(t_s + kHalf, r[1]);
          tmem_wait_frag(r);
          // ---- exponents: scores (times K's scales) less the rows'
          // references, masked, and the thread's largest; masked or not is two
          // bodies: a branch a value would leave no independent work between
          // the links of each value's chain
          const int first = t * T + col2;
          float top = -INFINITY;
          const auto exponents = [&](auto with_mask) {
            constexpr bool kMask = decltype(with_mask)::value;
            const uint64_t sc = pack_f2(x.scale, x.scale);
#pragma unroll
            for (int j = 0; j < T / 8; ++j) {
              uint64_t k2 = sc;
              if constexpr (kQuant) k2 = *reinterpret_cast<const uint64_t*>(sk + 8 * j);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t* v = &r[k >> 1][4 * j + 2 * (k & 1)];
                float2 u = unpack_f2(fma_f2(pack_f2(__uint_as_float(v[0]), __uint_as_float(v[1])), k2, pack_f2(nbase[k], nbase[k])));
                if constexpr (kMask) {
                  if (first + 8 * j < lo[k] || first + 8 * j >= hi[k]) u.x = -INFINITY;
                  if (first + 8 * j + 1 < lo[k] || first + 8 * j + 1 >= hi[k]) u.y = -INFINITY;
                }
                v[0] = __float_as_uint(u.x), v[1] = __float_as_uint(u.y);
                top = fmaxf(top, fmaxf(u.x, u.y));
              }
            }
          };
          if (t * T < all_lo || (t + 1) * T > all_hi) exponents(std::true_type{});
          else exponents(std::false_type{});
          // ---- references, see attn_lag
          constexpr float kLag = attn_lag<B>();
          float tile_e = 0.f;  // the largest exponent of the tile's V scales
          if constexpr (kQuant) {
            const int2 e2 = *reinterpret_cast<const int2*>(exps + 2 * (g & 3));
            tile_e = static_cast<float>(max(e2.x, e2.y) - 15);
          }
          if (__any_sync(0xffffffffu, !begun || top + tile_e > kLag)) {
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < T / 8; ++j) {
              float2 ex;
              if constexpr (kQuant) {
                ex = *reinterpret_cast<const float2*>(scales + (8 + (g & 3)) * T + col2 + 8 * j);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t* v = &r[k >> 1][4 * j + 2 * (k & 1)];
                float2 u = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
                if constexpr (kQuant) u = unpack_f2(add_f2(pack_f2(u.x, u.y), pack_f2(ex.x, ex.y)));
                mx[k] = fmaxf(mx[k], fmaxf(u.x, u.y));
              }
            }
            float f[4];
            bool any = false;
            begun = true;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
              mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2)) - nbase[k];  // the largest score and exponent
              const float m1 = mx[k] > m[k] + kLag ? mx[k] : m[k];  // m = -inf: mx, where anything is seen
              const float nb1 = m1 == -INFINITY ? 0.f : -m1;
              const bool moved = nb1 != nbase[k] && m[k] != -INFINITY;  // else the row's O is zeros, or not begun
              f[k] = moved ? exp2_fast(nb1 - nbase[k]) : 1.f;
              any |= moved;
              const uint64_t d2 = pack_f2(nb1 - nbase[k], nb1 - nbase[k]);
#pragma unroll
              for (int j = 0; j < T / 8; ++j) {
                uint32_t* v = &r[k >> 1][4 * j + 2 * (k & 1)];
                const float2 u = unpack_f2(add_f2(pack_f2(__uint_as_float(v[0]), __uint_as_float(v[1])), d2));
                v[0] = __float_as_uint(u.x), v[1] = __float_as_uint(u.y);
              }
              m[k] = m1;
              nbase[k] = nb1;
              begun &= m1 != -INFINITY;
              sum[k] = mul_f2(sum[k], pack_f2(f[k], f[k]));
            }
            if (t > t0 && __any_sync(0xffffffffu, any)) {
              // P V of the tile before has to be over before O is touched
              ok = mbar_wait_warp(pv_done(g - 1), phase4(g - 1), abort_flag, a);
              if (!ok) break;
              tc_after();
#pragma unroll 2
              for (int c = 0; c < D / 16; ++c) {  // few registers: the scores stay where they are
                tmem_scale16(t_o + 16 * c, f[0], f[1]);
                tmem_scale16(t_o + kHalf + 16 * c, f[2], f[3]);
              }
              tmem_wait_st();
            }
          }
          // ---- weights, to where the scores were
          {
            uint32_t out[2][16];
#pragma unroll
            for (int j = 0; j < T / 8; ++j) {
              uint64_t v2 = 0;
              if constexpr (kQuant) v2 = *reinterpret_cast<const uint64_t*>(sv + 8 * j);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t* v = &r[k >> 1][4 * j + 2 * (k & 1)];
                uint64_t u = pack_f2(exp2_fast(__uint_as_float(v[0])), exp2_fast(__uint_as_float(v[1])));
                sum[k] = add_f2(sum[k], u);
                if constexpr (kQuant) u = mul_f2(u, v2);
                const float2 e = unpack_f2(u);
                out[k >> 1][2 * j + (k & 1)] = half2_bits(e.x, e.y);
              }
            }
            tmem_st_pairs(t_s, out[0]);
            tmem_st_pairs(t_s + kHalf, out[1]);
          }
          tmem_wait_st();
          tc_before();
          mbar_arrive(w_full(s, buf));
        }
        if (ok) {
          ok = mbar_wait_warp(pv_done(g - 1), phase4(g - 1), abort_flag, a);
          tc_after();
        }
      } else if (works) {
        // An M tile without rows: the warps say that they have seen each tile's
        // scores, and the scores two tiles on wait for that by way of P V. A
        // warp that only watched could fall four tiles behind, and wait for a
        // phase that has gone by.
        const int n = p.t1 - p.t0;
        for (int t = 0; t < n && ok; ++t, ++g) {
          ok = mbar_wait_warp(s_full(g), phase4(g), abort_flag, a);
          if (ok) mbar_arrive(w_full(s, g & 1));
        }
      }
      // the statistics of the thread's row `lane` of the warp: slot lane / 8 of
      // the lanes from 4 (lane % 8)
      float row_l = 0.f, row_base = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v2 = unpack_f2(sum[k]);
        float v = v2.x + v2.y;
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        const float a1 = __shfl_sync(0xffffffffu, v, 4 * (lane & 7)), b1 = __shfl_sync(0xffffffffu, -nbase[k], 4 * (lane & 7));
        if ((lane >> 3) == k) row_l = a1, row_base = b1;
      }
      // ---- epilogue: a thread holds its row's D values
      const int c0 = p.whole ? 0 : attn_cta_of(state.s, p.first), c1 = p.whole ? 0 : attn_cta_of(state.s, p.first + p.u.tiles - 1);
      if (active && ok) {
        const bool has = row < p.u.rows;
        int token = 0, head = 0;
        if (has) attn_row_of(a, p, row, token, head);
        float* slot = p.whole ? nullptr : attn_slot(a, blockIdx.x, static_cast<int>(blockIdx.x) == c0, C::kFloats);
        const float inv = !p.whole ? 1.f : row_l != 0.f ? 1.f / row_l : 0.f;
        // where the lane's row goes
        const unsigned long long out =
            p.whole ? reinterpret_cast<unsigned long long>(a.out.data + token * a.out.token_stride + head * a.out.head_stride)
                    : reinterpret_cast<unsigned long long>(slot + row * D);
        // Rows go out through shared memory, 64 bytes of each at a time, so
        // that four lanes write 64 neighbouring bytes of a row and a store
        // touches 8 lines and not 32 (a unit's rows took 8500 cycles that way).
        const uint32_t stage = sbase + C::kOffStage + (s * 4 + (warp & 3)) * 2048;
        const uint32_t put = stage + lane * 64, put_x = (lane >> 1) & 3;
        const bool whole = p.whole;
        const int last = min(32, p.u.rows - row0);  // rows of the warp
        // the rows that the lane writes a quarter of, and its places in them
        const int get_row = lane >> 2, get_ch = lane & 3;
        unsigned long long to[4];
        uint32_t get[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 8 * i + get_row;
          to[i] = __shfl_sync(0xffffffffu, out, rr) + 16 * get_ch;
          get[i] = stage + rr * 64 + ((get_ch ^ ((rr >> 1) & 3)) << 4);
        }
        const auto flush = [&](int byte) {  // the staged 64 bytes to byte `byte` of each row
          uint4 v[4];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                         : "r"(get[i]));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (8 * i + get_row < last) *reinterpret_cast<uint4*>(to[i] + byte) = v[i];
          __syncwarp();
        };
        uint32_t r[2][32];
        tmem_ld32(t_o, r[0]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          tmem_wait_ld(r[c & 1]);
          if (c + 1 < D / 32) tmem_ld32(t_o + 32 * (c + 1), r[(c + 1) & 1]);
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            // 0 4 1 5 2 6 3 7 back to the dims' order
            const int at = kPairs ? (i & ~7) + 2 * (i & 3) + ((i >> 2) & 1) : i;
            y[i] = row_l != 0.f ? __uint_as_float(r[c & 1][at]) * inv : 0.f;
          }
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sts128(put + ((i ^ put_x) << 4), half2_bits(y[8 * i], y[8 * i + 1]), half2_bits(y[8 * i + 2], y[8 * i + 3]),
                     half2_bits(y[8 * i + 4], y[8 * i + 5]), half2_bits(y[8 * i + 6], y[8 * i + 7]));
            flush(64 * c);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sts128(put + ((i ^ put_x) << 4), __float_as_uint(y[16 * h + 4 * i]), __float_as_uint(y[16 * h + 4 * i + 1]),
                       __float_as_uint(y[16 * h + 4 * i + 2]), __float_as_uint(y[16 * h + 4 * i + 3]));
              flush(128 * c + 64 * h);
            }
          }
        }
        if (has) {
          if (p.whole)
            attn_store_lse(a, token, head, row_base, row_l);
          else
            slot[C::kRows * D + row] = row_base, slot[C::kRows * D + C::kRows + row] = row_l;
        }
        tc_before();  // the next unit's first P V, ordered by its weights, overwrites O
        if constexpr (!kQuant) {
          if (cleaned[state.number & 3] == state.number && row < p.u.rows)
            put_back_row<D, C::kFloats>(a, p, row, static_cast<int>(blockIdx.x) == c0);
        }
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

  // nothing may be in flight when tensor memory is freed
  if (warp == kScoreWarp)
    for (int i = 0; i < 1 + C::kStreams; ++i)
      for (int r = 0; r < a.wait_limit; ++r)
        if (__all_sync(0xffffffffu, mbar_try_wait(drain + 8 * i, 0))) break;
  tc_before();
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------- host

template <int B, int D>
exq_status launch(const AttnCall& call, const AttnArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<B, D>;
  Maps maps;
  constexpr int kPart = B == 16 ? 128 : C::Packed::kPartBytes;
  constexpr CUtensorMapSwizzle kSwizzle = B == 6        ? CU_TENSOR_MAP_SWIZZLE_NONE
                                          : kPart == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                          : kPart == 64  ? CU_TENSOR_MAP_SWIZZLE_64B
                                                         : CU_TENSOR_MAP_SWIZZLE_32B;
  if (!split::encode_cache(&maps.k, a.codes[0], *call.cache, kPart / 4, kSwizzle) ||
      !split::encode_cache(&maps.v, a.codes[1], *call.cache, kPart / 4, kSwizzle))
    return EXQ_ERR_CUDA;
  const Extra x{std::fmax(std::fabs(a.scale_log2), 0x1p-126f), a.scale_log2 < 0};
  auto fn = attn_chunk_kernel<B, D>;
  static PerDevice state;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || !state.once(dev, [&] {
        cudaFuncAttributes at{};
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) == cudaSuccess &&
               cudaFuncGetAttributes(&at, fn) == cudaSuccess && (at.numRegs + 7) / 8 * 8 == kLaunchRegs;
      }))
    return EXQ_ERR_CUDA;
  fn<<<std::min(sms, kAttnMaxCtas), kThreads, C::kSmem, stream>>>(maps, a, x);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

template <int B>
exq_status launch_bits(const AttnCall& call, const AttnArgs& a, int sms, cudaStream_t stream) {
  switch (call.cache->D) {
    case 64: return launch<B, 64>(call, a, sms, stream);
    case 128: return launch<B, 128>(call, a, sms, stream);
    default: return launch<B, 256>(call, a, sms, stream);
  }
}

inline int rows_of(int D) { return D == 256 ? 128 : 256; }

}  // namespace chunk

exq_status launch_attn_chunk4(const AttnCall& c, const AttnArgs& a, int sms, cudaStream_t stream);
exq_status launch_attn_chunk6(const AttnCall& c, const AttnArgs& a, int sms, cudaStream_t stream);
exq_status launch_attn_chunk8(const AttnCall& c, const AttnArgs& a, int sms, cudaStream_t stream);
exq_status launch_attn_chunk16(const AttnCall& c, const AttnArgs& a, int sms, cudaStream_t stream);

}  // namespace exq
