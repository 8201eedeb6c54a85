// Products of a few fp16 rows with matrices of the microscaled 4-bit format on
// the block-scaled tcgen05 tensor cores: the decode product (one matrix) and
// the two products of an expert layer.
//
//   out[t][n] = sum_k x[t][k] w[n][k],   t < 16
//
// Every code is read once, so the floor is the codes' and scales' bytes. At
// 6.8 TB/s an SM gets some 40 codes a clock: turning them into fp16 in registers
// costs more instructions than it has (a first kernel on mma.sync reached 2.4
// TB/s, its integer pipe full). So the codes are never turned into anything:
// the tensor cores multiply them as they are, and x is brought to their form.
//
// A row of x as eight 4-bit rows: with s a power of two, |x| <= 4 s for all of
// a block, part 0 is the e2m1 number nearest to q = x / s, part p + 1 that
// nearest to 8 times what part p left, and
//   x = s (p0 + p1 / 8 + p2 / 64 + ...)
// e2m1's steps up to 4 are at most 1, so that at most 1/2 is left, times 8 at
// most 4 again: every step is exact in fp32, and after eight parts at most
// 2^-23 of the block's bound is left. The eight rows share their scales, lie
// beside one another as columns of the product, and the epilogue adds them
// with weights 8^-p. 16 tokens are 128 columns: a third of what the tensor
// cores could do while the codes arrive.
//
// Work is cut into units of 128 rows x 256 k of one matrix (16 KB of codes, 2
// or 1 KB of scales). The units of a call, those of one output tile in a row,
// are divided evenly over the CTAs, one an SM: no wave is left part-filled.
//
//   warp 0     brings a unit's codes, as one 2-D box (128-byte rows, 128-byte
//              swizzle), and its scale tiles, as one copy.
//   warp 6     brings the tokens' parts and their scales (a warp of its own:
//              behind the weights' copies theirs cost 250 ns a unit).
//              Few rows are split here, and there is no launch before this one
//              that does it: by warps 6 and 11-13, a row of a unit each; if x
//              is one row, by warps 6 and 11, a unit each.
//   warps 7-10 write a unit's scales to tensor memory, from shared memory by
//              way of registers. (The tensor core's own copy, tcgen05.cp, takes
//              55 clocks a tile and keeps MMAs waiting: 720 clocks a unit for
//              E4M3, of the 800 in which its codes arrive, and more for several
//              tokens of an expert.)
//   warp 1     issues the MMAs (M = 128 rows of the matrix, N = 8 columns a
//              token, K = 64).
//   warps 2-5  drain the sums: a lane is a row of the matrix.
//
// A tile whose units lie in several CTAs goes through the workspace: each
// writes its part, the last to arrive (a counter) adds them in CTA order, so
// that the result does not depend on who it is.
//
// One row of 28672 x 8192, E8M0: 25.5 us (4.9 TB/s; 6.4 while it streams), of
// 4096 x 4096: 7.9 us, which is set-up, the first bytes' way and the last sums';
// sixteen rows of 28672 x 8192, E4M3: 29 us. Experts: 5 tokens of 8 of 128 of
// 1536 x 4096, E4M3, 84.4 us (4.4 TB/s, 7 while gate and up stream).
#pragma once

#include "exq_fp4.cuh"

namespace exq {
namespace fp4s {

static __device__ unsigned g_stream_err;

enum Mode { kGemv = 0, kUp = 1, kDown = 2 };

constexpr int kRows = 128;           // rows of a unit: the MMA's M
constexpr int kUnitK = 256;          // k of a unit: 128 bytes of codes a row
// of a CTA: the warps above
__host__ __device__ constexpr int threads_of(int NT, bool here) { return 32 * (!here ? 11 : NT == 1 ? 12 : 14); }
constexpr int kParts = 8;            // 4-bit rows of a row of x
constexpr int kMaxTokens = 16;
constexpr int kMaxPairs = 256;       // tokens x experts of each
constexpr int kMaxExperts = 512;
constexpr int kMaxStages = 10;

// a stage: codes, scale tiles, the tokens' parts and their scales
constexpr int kOffScales = kRows * kUnitK / 2;
constexpr int kOffX = kOffScales + 2048;
static_assert(kOffX % 1024 == 0, "swizzle atoms");
// The decode product takes all tokens: the parts are a matrix of 8 M rows with
// its scale tiles. An expert's tokens are picked one by one: a token's parts
// of a unit are a piece, written as shared memory has it: the 8 rows of 128
// bytes, swizzled, then for each scale tile 8 lines of 16 bytes, a line a row,
// its first word the scales. Four pieces' lines are 32, a lane each, so that
// MMAs are made for up to four tokens at a time.
constexpr int kLines = 8 * 16;
constexpr int kSlot = 2048;          // of a piece in a stage
__host__ __device__ constexpr int unit_tiles(int fmt) { return kUnitK / fp4_tile_k(fmt); }
__host__ __device__ constexpr int piece_bytes(int fmt) { return 1024 + unit_tiles(fmt) * kLines; }
// byte of the word of 8 codes at k (a multiple of 8, in the unit) of part p
__host__ __device__ constexpr int piece_word(int p, int k) { return p * 128 + (((k / 32) ^ p) * 16) + (k % 32) / 2; }

constexpr int kSmemTotal = 222 * 1024;  // (room is left for a CTA of the small kernels before and after)
constexpr int kRest = 20 * 1024;     // barriers, the experts' tables, sums, alignment
constexpr int kRing = kSmemTotal - kRest;

constexpr uint32_t kTmemCols = 512;
constexpr int kMaxBuffers = 4;

// Scale of a block of x: 2^(e - 1) for a largest magnitude in [2^e, 2^(e + 1)).
// An e4m3 scale has 18 powers of two: for fp16 the largest is 2^14 (times 2^-6
// that is 2^8, e4m3's largest power), and a block whose scale would be under
// the smallest takes that one, 2^-3: its eighth part counts 2^-25 then, half of
// fp16's smallest number. What lies between an expert's products (h) is
// divided by a power of two first that brings a token's largest to [1, 2) (below
// 2^-100: by 2^-100): the smallest scale is 2^-18 then, and 2^-40 is left of it.
constexpr int kXTop = 14, kHTop = -1;          // exponents of the largest scales
__host__ __device__ constexpr int e4m3_shift(int top) { return top - 8; }

struct Args {
  const uint8_t* sc0;      // scale tiles of the matrix, or of expert 0's gate or down
  const uint8_t* sc1;      // of expert 0's up
  size_t sc_stride;        // from expert to expert
  const uint8_t* x;        // gemv: scale tiles of the parts; else pieces [token or pair, unit]
  const uint16_t* rows_of_x;  // gemv that splits x: [M, K]
  uint16_t* y;             // [M, rows] (not up)
  float* h;                // up: [pairs, rows]
  unsigned* h_most;        // [pairs]: bits of the largest finite magnitude of h
  const float *f0, *f1;    // experts' factors of gate and up, or of down, or NULL
  const int32_t* ids;      // [M, top_k]
  const float* weights;
  unsigned* counters;
  float* part;             // [CTAs][2][part_floats]
  float factor;
  int rows, K, M;
  int row_tiles, k_units, k_tiles;
  int top_k, n_experts, act;
  // up: the down product that follows
  const uint8_t* down_scales;
  size_t down_stride;
  int down_row_tiles, down_k_units, down_k_tiles;
  int wait_limit, starve;
};

// Between the last of up's codes and the first of down's the SMs wait for sums,
// for h's parts and for a set-up, some 10 us. Up's CTAs ask for down's first
// units meanwhile, as far as L2 (this many a CTA: 44 MB in all).
constexpr int kAhead = 16;

// floats of one CTA's part of a tile: a value for each row, token (and matrix)
__host__ __device__ constexpr int part_floats(int mode) { return kRows * kMaxTokens * (mode == kUp ? 2 : 1); }

// The experts of a call, the same in every CTA: those that some token chose,
// ascending, with the tokens of each and the place of (expert, token) in ids.
struct Experts {
  int n, most_tokens, pad[2];
  int expert[kMaxPairs];
  unsigned tokens[kMaxPairs];                 // a bit each
  uint8_t place[kMaxPairs][kMaxTokens];       // the first, where an id repeats
  int ids[kMaxPairs];
  float weight[kMaxPairs];                    // by that place: those of an id that repeats are added up
};
static_assert(sizeof(Experts) + kRows * kMaxTokens * 4 + 512 + 1024 <= kRest, "shared memory budget");

// ---------------------------------------------------------------- parts

// The e-1 of a block's scale 2^(e-1) from the bits of its largest magnitude
// (fp32, finite), and the byte that the format has for it.
template <int FMT>
__device__ __forceinline__ int part_exponent(float most, int top) {
  const int e = static_cast<int>(__float_as_uint(most) >> 23) - 128;  // -128 for zero and subnormals
  if constexpr (FMT == EXQ_FP4_E4M3) return min(max(e, top - 17), top);
  return max(e, -126);
}

template <int FMT>
__device__ __forceinline__ uint32_t part_scale_byte(int e, int top) {
  if constexpr (FMT == EXQ_FP4_E8M0) return static_cast<uint32_t>(e + 127);
  const int p = e - e4m3_shift(top);  // -9 .. 8
  return p >= -6 ? static_cast<uint32_t>(p + 7) << 3 : 1u << (p + 9);
}

// h's power of two: e of [2^e, 2^(e + 1)) for the largest magnitude, given as bits
__device__ __forceinline__ int h_exponent(unsigned most) { return max(static_cast<int>(most >> 23) - 127, -100); }

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// what h is multiplied by: 2^-e, for e = 127 a subnormal number
__device__ __forceinline__ float h_scale(unsigned most) {
  const int e = h_exponent(most);
  return e == 127 ? __uint_as_float(0x00400000u) : pow2(-e);
}

// Eight values of a row as words of codes of the parts, and the scale word
// that they share with the 8 (E4M3) or 16 threads of four blocks; `c` counts
// the threads along the row. By whole warps.
template <int FMT>
__device__ __forceinline__ void split8(float (&q)[8], int top, int c, uint32_t (&words)[kParts], uint32_t& scales) {
  constexpr int kBlockThreads = fp4_block(FMT) / 8, kWordThreads = 4 * kBlockThreads;
  uint32_t m = 0u;  // bits of the block's largest magnitude (infinity and NaN are above all others)
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(q[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < kBlockThreads; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  const bool bad = m >= 0x7F800000u;  // the block is NaN
  const int e = bad ? 0 : part_exponent<FMT>(__uint_as_float(m), top);
  const uint32_t byte = bad ? (FMT == EXQ_FP4_E4M3 ? 0x7Fu : 0xFFu) : part_scale_byte<FMT>(e, top);
  const float r = pow2(-e);
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = bad ? 0.f : q[j] * r;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    words[p] = e2m1x8(q);
    const uint32_t v[4] = {e2m1x2_f16<0>(words[p]), e2m1x2_f16<1>(words[p]), e2m1x2_f16<2>(words[p]), e2m1x2_f16<3>(words[p])};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
      q[2 * j] = (q[2 * j] - d.x) * 8.f;
      q[2 * j + 1] = (q[2 * j + 1] - d.y) * 8.f;
    }
  }
  scales = byte << (8 * ((c / kBlockThreads) & 3));
#pragma unroll
  for (int d = kBlockThreads; d < kWordThreads; d <<= 1) scales |= __shfl_xor_sync(0xffffffffu, scales, d);
}

// eight fp16 numbers
__device__ __forceinline__ void to_f32(uint4 x, float (&q)[8]) {
  const uint32_t h[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    q[2 * j] = v.x;
    q[2 * j + 1] = v.y;
  }
}

// ---------------------------------------------------------------- tcgen05

// K-major, 128-byte swizzle, 8-row groups `stride` bytes apart
__device__ __forceinline__ uint64_t codes_desc(uint32_t addr, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (static_cast<uint64_t>(stride >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ uint32_t idesc_for(int fmt, int n) {  // e2m1 operands, K-major, M = 128
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((fmt == EXQ_FP4_E8M0 ? 1u : 0u) << 23) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

template <int FMT>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                           uint32_t accumulate) {
  if constexpr (FMT == EXQ_FP4_E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
}

// four scale tiles (16 bytes of each for the lane) to 16 columns of this warp's lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint4 (&t)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(t[0].x), "r"(t[0].y), "r"(t[0].z), "r"(t[0].w), "r"(t[1].x), "r"(t[1].y), "r"(t[1].z), "r"(t[1].w),
        "r"(t[2].x), "r"(t[2].y), "r"(t[2].z), "r"(t[2].w), "r"(t[3].x), "r"(t[3].y), "r"(t[3].z), "r"(t[3].w)
      : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of this warp's lanes, there after wait_ld of the same registers: several may be on their way
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void wait_ld(float (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])::"memory");
}

// a token's sum from those of its parts
__device__ __forceinline__ float join_parts(const float* d) {
  float v = d[7];
#pragma unroll
  for (int p = 6; p >= 0; --p) v = fmaf(v, 0.125f, d[p]);
  return v;
}

// ---------------------------------------------------------------- experts

// The experts' tables, by all threads of the CTA.
__device__ __forceinline__ void find_experts(const Args& a, Experts* e, unsigned* used, bool report) {
  const int tid = threadIdx.x, pairs = a.M * a.top_k;
  if (tid < kMaxExperts / 32) used[tid] = 0u;
  const int id = tid < pairs ? __ldcg(a.ids + tid) : -1;
  const float weight = tid < pairs ? __ldcg(a.weights + tid) : 0.f;
  if (tid < kMaxPairs) {
    e->tokens[tid] = 0u;
    e->ids[tid] = id;
    e->weight[tid] = weight;
  }
  __syncthreads();
  const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(a.n_experts);
  if (good) atomicOr(&used[id >> 5], 1u << (id & 31));
  if (report && id != -1 && !good) atomicOr(&g_stream_err, kDevErrBadExpert);
  __syncthreads();
  if (tid == 0) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) n += __popc(used[i]);
    e->n = n;
    e->most_tokens = 1;
  }
  bool first = good;
  float sum = 0.f;
  int slot = 0;
  if (good) {
    slot = __popc(used[id >> 5] & ((1u << (id & 31)) - 1u));
#pragma unroll
    for (int w = 0; w < kMaxExperts / 32; ++w) slot += w < (id >> 5) ? __popc(used[w]) : 0;
    e->expert[slot] = id;
    const int t = tid / a.top_k;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int p = min(t * a.top_k + j, kMaxPairs - 1);
      const bool same = e->ids[p] == id && j < a.top_k;
      const float w = e->weight[p];
      first = first && (!same || p >= tid);
      sum += same ? w : 0.f;
    }
    if (first) {
      e->place[slot][t] = static_cast<uint8_t>(tid);
      atomicOr(&e->tokens[slot], 1u << t);
    }
  }
  __syncthreads();
  if (first) {
    e->weight[tid] = sum;
    atomicMax(&e->most_tokens, __popc(e->tokens[slot]));
  }
  __syncthreads();
}
static_assert(kMaxPairs <= threads_of(1, false), "a place a thread");

// v times the logistic function of v, or of 2 u, which is (1 + tanh u) / 2: where u is
// very negative 1 + tanh u is a difference of two numbers near 1, and this is not.
// (__expf is off by 2 + |1.2 t| of its last bits: less than 2^-16 as far as t = -88,
// below which the result is zero.)
__device__ __forceinline__ float activate(float v, int act) {
  const float t = act == EXQ_ACT_SILU ? v : 1.5957691216057308f * (v + 0.044715f * v * v * v);
  return v / (1.f + __expf(-t));
}

// bit number j (from 0) that is set
__device__ __forceinline__ int nth_bit(unsigned m, int j) {
  for (; j > 0; --j) m &= m - 1u;
  return __ffs(static_cast<int>(m)) - 1;
}

// ---------------------------------------------------------------- units

// How many units a call has. `slots`: the experts, or one.
__device__ __forceinline__ long long units_of(const Args& a, int slots) {
  return static_cast<long long>(a.row_tiles) * a.k_units * slots;
}

// A unit's place: its expert (the index in Experts), tile of rows and k. The
// division is made once a CTA; from unit to unit the place counts up.
template <int MODE>
struct Place {
  int kc, slot, row;

  __device__ __forceinline__ Place(const Args& a, int experts, long long u) {
    const long long q = u / a.k_units;
    kc = static_cast<int>(u - q * a.k_units);
    slot = 0;
    row = static_cast<int>(q);
    if constexpr (MODE == kUp) {
      slot = static_cast<int>(q / a.row_tiles);
      row = static_cast<int>(q) - slot * a.row_tiles;
    } else if constexpr (MODE == kDown) {
      row = static_cast<int>(q / max(experts, 1));  // (without experts there is no unit)
      slot = static_cast<int>(q) - row * experts;
    }
  }

  // the last unit of its tile
  __device__ __forceinline__ bool ends(const Args& a, int experts) const {
    return kc + 1 == a.k_units && (MODE != kDown || slot + 1 == experts);
  }

  __device__ __forceinline__ void next(const Args& a, int experts) {
    if (++kc < a.k_units) return;
    kc = 0;
    if constexpr (MODE == kDown) {
      if (++slot < experts) return;
      slot = 0;
      ++row;
    } else {
      if (++row < a.row_tiles || MODE == kGemv) return;
      row = 0;
      ++slot;
    }
  }
};

// CTA b of `ctas` that divide n units has those from first_unit(b) up to
// first_unit(b + 1); `owner` is the one that has unit u.
__host__ __device__ __forceinline__ long long first_unit(int b, long long n, int ctas) { return b * n / ctas; }

__host__ __device__ __forceinline__ int owner(long long u, long long n, int ctas) {
  if (n * ctas < (1LL << 31)) return (static_cast<int>(u + 1) * ctas - 1) / static_cast<int>(n);
  return static_cast<int>(((u + 1) * ctas - 1) / n);
}

// counts stages or buffers, and the parity of their barriers
struct Turn {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      parity ^= 1u;
    }
  }
};

// v[w][j] becomes the sum of part j (of n) of matrix w of CTAs b0 .. b1, in their order; several parts' loads are in flight at a
// time. OWN: this CTA's part is what v has; else it is read like the others, which takes fewer registers: the few-row product is
// to leave room for the next call's small kernel (13 x 4096 x 11008: 13.0 us with 128 registers, 15.5 with 140), and with
// sixteen tokens an expert's products lost by it what they gained.
template <bool OWN, int W, int N, typename PartOf>
__device__ __forceinline__ void add_parts(float (&v)[W][N], int n, int b0, int b1, PartOf part_of) {
  constexpr int kAtOnce = W * N > 32 ? 2 : W * N > 8 ? 4 / W : 8;
  const int me = OWN ? static_cast<int>(blockIdx.x) : -1;
  float own[W][N];
#pragma unroll
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (OWN) own[w][j] = v[w][j];
      v[w][j] = 0.f;
    }
  for (int b = b0; b <= b1; b += kAtOnce) {
    float t[kAtOnce][W][N];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const bool load = !OWN || b + i != me;
      const float* p = part_of(min(b + i, b1));
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int j = 0; j < N; ++j) t[i][w][j] = load && j < n ? __ldcg(p + (w * kMaxTokens + j) * kRows) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (b + i <= b1) {
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
          for (int j = 0; j < N; ++j) v[w][j] += OWN && b + i == me ? own[w][j] : t[i][w][j];
      }
  }
}

// NT: rows of x, at most. (What drains the sums is unrolled over them, and in a
// short call most of its code is fetched for the first time: one row's is a
// sixteenth of sixteen's.)
// HERE: x's rows, or the one row of h of an expert, are split in this kernel.
template <int FMT, int MODE, int NT, bool HERE>
__global__ void __launch_bounds__(threads_of(NT, HERE), 1)
    stream_kernel(const __grid_constant__ CUtensorMap m0, const __grid_constant__ CUtensorMap m1,
                  const __grid_constant__ CUtensorMap mx, const __grid_constant__ Args a) {
  constexpr int kMatrices = MODE == kUp ? 2 : 1;  // of a unit, a stage each
  constexpr int kVals = NT < 2 ? 2 : NT;           // values of a lane (two tokens' come at a time)
  constexpr bool kOwn = MODE != kGemv && NT <= 8;
  constexpr int kTiles = unit_tiles(FMT), kThreads = threads_of(NT, HERE);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sums = reinterpret_cast<float*>(smem + kRing);                 // down: [tokens][rows]
  uint64_t* full = reinterpret_cast<uint64_t*>(sums + kRows * kMaxTokens);
  uint64_t* empty = full + kMaxStages;
  uint64_t* ready = empty + kMaxStages;  // and the scales are in tensor memory
  uint64_t* dfull = ready + kMaxStages;
  uint64_t* dempty = dfull + kMaxBuffers;
  uint64_t* done = dempty + kMaxBuffers;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last = abort_flag + 1;
  volatile int* there = last + 1;  // (a word of its own: `last` may still be read, of the tile before)
  unsigned* used = reinterpret_cast<unsigned*>(tmem_slot + 4);
  Experts* ex = reinterpret_cast<Experts*>(used + kMaxExperts / 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1 + (HERE && NT > 1 ? 4 : 1));  // the weights' copies and x's parts
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&ready[s]), 4);
    }
    for (int b = 0; b < kMaxBuffers; ++b) {
      mbar_init(smem_u32(&dfull[b]), 1);
      mbar_init(smem_u32(&dempty[b]), 4);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && elect_one()) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&m0)) : "memory");
    if constexpr (MODE == kUp) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&m1)) : "memory");
    if constexpr (MODE != kDown) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mx)) : "memory");
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if constexpr (MODE == kUp) {
    // ids and weights may come from the launch before
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  if constexpr (MODE == kGemv && HERE) asm volatile("griddepcontrol.wait;" ::: "memory");  // w may come from the launch before
  if constexpr (MODE != kDown) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n_experts = 1, most_tokens = a.M;
  if constexpr (MODE != kGemv) {
    find_experts(a, ex, used, MODE == kUp && blockIdx.x == 0);
    n_experts = ex->n;
    most_tokens = ex->most_tokens;
  }
  const long long n_units = units_of(a, n_experts);
  if constexpr (MODE == kDown) {
    if (n_units == 0) {  // no token has an expert
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const long long n = static_cast<long long>(a.M) * a.rows;
      for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n;
           i += static_cast<long long>(gridDim.x) * kThreads)
        a.y[i] = 0;
    }
  }
  const int ctas = static_cast<int>(n_units < gridDim.x ? n_units : gridDim.x);
  const long long u0 = ctas > 0 ? first_unit(blockIdx.x, n_units, ctas) : 0;
  const int n_mine = static_cast<int>(blockIdx.x) < ctas ? static_cast<int>(first_unit(blockIdx.x + 1, n_units, ctas) - u0) : 0;

  // the ring and the buffers of sums go by the most tokens that a matrix of the call has
  const int off_xs = kOffX + 1024 * most_tokens;                        // gemv: the parts' scale tiles
  const int stage_bytes = MODE == kGemv ? off_xs + 2048 : kOffX + kSlot * ((most_tokens + 3) / 4 * 4);
  const int n_stages = min(kMaxStages, kRing / stage_bytes);
  const int cols = (8 * most_tokens + 15) / 16 * 16;                    // of one sum
  const int buffer_cols = cols * kMatrices;
  // tensor memory: the buffers, then places for the scales of stages (16 columns of the matrix's, 16 for each four tokens);
  // three of them at least, while there are two buffers or one
  const int groups = MODE == kGemv ? 1 : (most_tokens + 3) / 4;
  const int scale_cols = 16 + 16 * groups;
  const int n_buffers = max(1, min(kMaxBuffers, (static_cast<int>(kTmemCols) - 3 * scale_cols) / buffer_cols));
  const int n_places = min(n_stages, (static_cast<int>(kTmemCols) - n_buffers * buffer_cols) / scale_cols);

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned everyone = MODE == kGemv ? (1u << a.M) - 1u : 0u;

  if (warp == 0) {
    // ------------------------------------------------------------ codes and scales of the matrix
    const bool leader = elect_one();
    int issued = 0;
    if (!a.starve) {  // test hook: starved producers issue nothing
      Place<MODE> at(a, n_experts, u0);
      Turn turn;
      bool ok = true;
      for (int left = n_mine; left > 0 && ok; --left) {
        const int id = MODE == kGemv ? 0 : ex->expert[at.slot];
        const uint32_t sb = min(kTiles, a.k_tiles - at.kc * kTiles) * 512;
        const size_t off = id * a.sc_stride + (static_cast<size_t>(at.row) * a.k_tiles + at.kc * kTiles) * 512;
#pragma unroll
        for (int which = 0; which < kMatrices; ++which) {
          if (!mbar_wait_warp(smem_u32(&empty[turn.i]), turn.parity ^ 1u, abort_flag, a.wait_limit, &g_stream_err)) {
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t st = smem_u32(smem) + turn.i * stage_bytes, bar = smem_u32(&full[turn.i]);
            mbar_expect_tx(bar, kOffScales + sb);
            tma_load_2d(st, which == 0 ? &m0 : &m1, at.kc * (kUnitK / 2), id * a.rows + at.row * kRows, bar);
            bulk_load(st + kOffScales, (which == 0 ? a.sc0 : a.sc1) + off, sb, bar);
          }
          __syncwarp();
          turn.next(n_stages);
          ++issued;
        }
        at.next(a, n_experts);
      }
      if constexpr (MODE == kUp) {
        Args d;
        d.row_tiles = a.down_row_tiles;
        d.k_units = a.down_k_units;
        const long long n_down = units_of(d, n_experts);
        const int down_ctas = static_cast<int>(n_down < gridDim.x ? n_down : gridDim.x);
        if (static_cast<int>(blockIdx.x) < down_ctas) {
          const long long d0 = first_unit(blockIdx.x, n_down, down_ctas);
          const int n = min(kAhead, static_cast<int>(first_unit(blockIdx.x + 1, n_down, down_ctas) - d0));
          Place<kDown> to(d, n_experts, d0);
          for (int i = 0; i < n; ++i) {
            if (leader) {
              const int id = ex->expert[to.slot];
              asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&mx)),
                           "r"(to.kc * (kUnitK / 2)), "r"(id * a.K + to.row * kRows) : "memory");
              asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(
                               a.down_scales + id * a.down_stride + (static_cast<size_t>(to.row) * a.down_k_tiles + to.kc * kTiles) * 512)),
                           "r"(min(kTiles, a.down_k_tiles - to.kc * kTiles) * 512) : "memory");
            }
            __syncwarp();
            to.next(d, n_experts);
          }
        }
      }
    }
    await_issued(full, issued, n_stages, a.wait_limit);
  } else if (HERE && (warp == 6 || warp > 10)) {
    // ------------------------------------------------------------ rows to parts
    if constexpr (MODE == kDown) asm volatile("griddepcontrol.wait;" ::: "memory");  // for h
    if (!a.starve) {
      constexpr int kWordThreads = fp4_tile_k(FMT) / 8;
      constexpr int kMost = (NT + 3) / 4;  // rows of a unit for a warp
      const int group = warp == 6 ? 0 : warp - 10;
      Place<MODE> at(a, n_experts, u0);
      Turn turn;
      int left = n_mine;
      // Of one row each warp takes the units of every second place. (Every second unit would not do: with an odd number of
      // stages a warp would come to a place every second time round, and a barrier's parity would tell it nothing.)
      auto step = [&]() {
        do {
          at.next(a, n_experts);
          turn.next(n_stages);
          --left;
        } while (NT == 1 && left > 0 && (turn.i & 1) != group);
      };
      int before = 0;  // rows of the units before: they go to the warps in turn
      uint4 next[kMost][MODE == kGemv ? 1 : 2];  // (taken apart when it is there, not here)
      unsigned most[kMost];
      int mine = 0;    // the first row of this warp, of the unit that `next` is of
      auto load = [&]() {
        mine = NT == 1 ? 0 : (group - before) & 3;
        before += a.M;
        const int k = at.kc * kUnitK + 8 * lane;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const int t = mine + 4 * i;
          const bool in = t < a.M && k < a.K;
          const uint4 none = make_uint4(0u, 0u, 0u, 0u);
          if constexpr (MODE == kGemv) {
            next[i][0] = in ? __ldg(reinterpret_cast<const uint4*>(a.rows_of_x + static_cast<size_t>(t) * a.K + k)) : none;
          } else {
            const int pair = ex->place[at.slot][0];  // (of one token)
            const uint4* src = reinterpret_cast<const uint4*>(a.h + static_cast<size_t>(pair) * a.K + k);
            next[i][0] = in ? __ldcg(src) : none;
            next[i][1] = in ? __ldcg(src + 1) : none;
            most[i] = __ldcg(a.h_most + pair);
          }
        }
      };
      if (NT == 1 && group == 1) step();
      if (left > 0) load();
      while (left > 0) {
        float q[kMost][8];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          if constexpr (MODE == kGemv) {
            to_f32(next[i][0], q[i]);
          } else {
            const float r = h_scale(most[i]);
            const uint32_t b[8] = {next[i][0].x, next[i][0].y, next[i][0].z, next[i][0].w,
                                   next[i][1].x, next[i][1].y, next[i][1].z, next[i][1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) q[i][j] = __uint_as_float(b[j]) * r;
          }
        }
        const int t0 = mine;
        const Turn now = turn;
        step();
        if (left > 0) load();
        if (!mbar_wait_warp(smem_u32(&empty[now.i]), now.parity ^ 1u, abort_flag, a.wait_limit, &g_stream_err)) break;
        uint8_t* st = smem + now.i * stage_bytes;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const int t = t0 + 4 * i;
          if (t >= a.M) break;
          uint32_t words[kParts], scales;
          split8<FMT>(q[i], MODE == kDown ? kHTop : kXTop, lane, words, scales);
          uint8_t* piece = st + kOffX + t * 1024;
#pragma unroll
          for (int p = 0; p < kParts; ++p) *reinterpret_cast<uint32_t*>(piece + piece_word(p, 8 * lane)) = words[p];
          const int p = lane % kWordThreads, tile = lane / kWordThreads;  // a line of the scale tile for each part
          if (p < kParts)
            *reinterpret_cast<uint32_t*>(MODE == kGemv ? st + off_xs + tile * 512 + fp4_tile_byte(t * kParts + p)
                                                       : piece + 1024 + tile * kLines + p * 16) = scales;
        }
        if (t0 < a.M) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the tensor core reads it
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&full[now.i]));
      }
    }
  } else if (!HERE && warp == 6) {
    // ------------------------------------------------------------ the tokens' parts
    const bool leader = elect_one();
    int issued = 0;
    // they come from the launch before
    if constexpr (MODE != kUp) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!a.starve) {
      Place<MODE> at(a, n_experts, u0);
      Turn turn;
      bool ok = true;
      for (int left = n_mine; left > 0 && ok; --left) {
        const unsigned tokens = MODE == kGemv ? 0u : ex->tokens[at.slot];
        const int n_tok = __popc(tokens);
        const uint8_t* src = nullptr;  // lane: the piece of a token of the unit
        if (lane < n_tok) {
          const int token = nth_bit(tokens, lane);
          src = a.x + (static_cast<size_t>(MODE == kDown ? ex->place[at.slot][token] : token) * a.k_units + at.kc) * piece_bytes(FMT);
        }
#pragma unroll
        for (int which = 0; which < kMatrices; ++which) {
          if (!mbar_wait_warp(smem_u32(&empty[turn.i]), turn.parity ^ 1u, abort_flag, a.wait_limit, &g_stream_err)) {
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(smem) + turn.i * stage_bytes, bar = smem_u32(&full[turn.i]);
          if constexpr (MODE == kGemv) {
            if (leader) {
              const uint32_t sb = min(kTiles, a.k_tiles - at.kc * kTiles) * 512;
              mbar_expect_tx(bar, a.M * 1024 + sb);
              tma_load_2d(st + kOffX, &mx, at.kc * (kUnitK / 2), 0, bar);
              bulk_load(st + off_xs, a.x + static_cast<size_t>(at.kc) * kTiles * 512, sb, bar);
            }
          } else {
            if (leader) mbar_expect_tx(bar, n_tok * piece_bytes(FMT));
            __syncwarp();
            if (lane < n_tok) bulk_load(st + kOffX + lane * kSlot, src, piece_bytes(FMT), bar);
          }
          __syncwarp();
          turn.next(n_stages);
          ++issued;
        }
        at.next(a, n_experts);
      }
    }
    await_issued(full, issued, n_stages, a.wait_limit);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    Place<MODE> at(a, n_experts, u0);
    Turn turn, buf, place;
    bool fresh = true;  // the next unit begins a buffer
    bool ok = true;
    for (int left = n_mine; left > 0 && ok; --left) {
      const int tokens = MODE == kGemv ? 1 : __popc(ex->tokens[at.slot]);  // (all of x at once)
      const int n_k = min(4, (a.K - at.kc * kUnitK + 63) / 64);  // MMAs with k of the matrices
      const uint32_t d0 = tmem + buf.i * buffer_cols;
      if (fresh && !mbar_wait_warp(smem_u32(&dempty[buf.i]), buf.parity ^ 1u, abort_flag, a.wait_limit, &g_stream_err)) break;
#pragma unroll
      for (int which = 0; which < kMatrices; ++which) {
        if (!mbar_wait_warp(smem_u32(&ready[turn.i]), turn.parity, abort_flag, a.wait_limit, &g_stream_err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = smem_u32(smem) + turn.i * stage_bytes;
        const uint32_t sa = tmem + n_buffers * buffer_cols + place.i * scale_cols;
        const uint64_t ad = codes_desc(st, 1024);
        if (leader) {
          for (int g = 0; g < tokens; g += 4) {
            const uint32_t sb = sa + 16 + 4 * g, d = d0 + 8 * g + which * cols;
            const uint32_t idesc = idesc_for(FMT, MODE == kGemv ? cols : (8 * min(4, tokens - g) + 15) / 16 * 16);
            const uint64_t bd = codes_desc(st + kOffX + g * kSlot, MODE == kGemv ? 1024 : kSlot);
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 64 k: 32 bytes of a row
              if (j >= n_k) break;
              const bool first = j == 0 && fresh;
              if constexpr (FMT == EXQ_FP4_E4M3) {
                mma_scaled<FMT>(d, ad + 2 * j, bd + 2 * j, idesc, sa + 4 * j, sb + 4 * j, !first);
              } else {  // two scales of the tile's four: byte 0 or 2 of each word
                const uint32_t id = (j & 1) ? idesc | (2u << 4) | (2u << 29) : idesc;
                mma_scaled<FMT>(d, ad + 2 * j, bd + 2 * j, id, sa + 4 * (j >> 1), sb + 4 * (j >> 1), !first);
              }
            }
          }
        }
        __syncwarp();
        if (leader) commit(smem_u32(&empty[turn.i]));
        __syncwarp();
        turn.next(n_stages);
        place.next(n_places);
      }
      if (!ok) break;
      fresh = left == 1 || at.kc + 1 == a.k_units;  // the end of a tile, or (down) of an expert's share of it
      if (fresh) {
        if (leader) commit(smem_u32(&dfull[buf.i]));
        __syncwarp();
        buf.next(n_buffers);
      }
      at.next(a, n_experts);
    }
    // the MMAs are over before tensor memory is given back
    if (leader) commit(smem_u32(done));
    __syncwarp();
    for (int r = 0; r < a.wait_limit; ++r)
      if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(done), 0))) break;
  } else if (warp >= 7 && warp <= 10) {
    // ------------------------------------------------------------ scales to tensor memory
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Place<MODE> at(a, n_experts, u0);
    Turn turn, place, old;  // old: the stage whose MMAs read this place last
    int n = 0;
    bool ok = true;
    for (int left = n_mine; left > 0 && ok; --left) {
      const int tokens = MODE == kGemv ? 1 : __popc(ex->tokens[at.slot]);
#pragma unroll
      for (int which = 0; which < kMatrices; ++which) {
        if (!mbar_wait_warp(smem_u32(&full[turn.i]), turn.parity, abort_flag, a.wait_limit, &g_stream_err)) {
          ok = false;
          break;
        }
        const uint8_t* st = smem + turn.i * stage_bytes;
        uint4 t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = *reinterpret_cast<const uint4*>(st + kOffScales + j % kTiles * 512 + lane * 16);
        if (n_places < n_stages) {
          if (n >= n_places) {
            if (!mbar_wait_warp(smem_u32(&empty[old.i]), old.parity, abort_flag, a.wait_limit, &g_stream_err)) {
              ok = false;
              break;
            }
            old.next(n_stages);
          }
          ++n;
        }
        tc_fence_after();
        const uint32_t to = tmem + lanes + n_buffers * buffer_cols + place.i * scale_cols;
        tmem_st16(to, t);
        for (int g = 0; g < tokens; g += 4) {
          // all of x's, in tiles; or those of four tokens, a line a lane
          const uint8_t* from = MODE == kGemv ? st + off_xs + lane * 16
                                              : st + kOffX + (g + (lane >> 3)) * kSlot + 1024 + (lane & 7) * 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) t[j] = *reinterpret_cast<const uint4*>(from + j % kTiles * (MODE == kGemv ? 512 : kLines));
          tmem_st16(to + 16 + 4 * g, t);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ready[turn.i]));
        turn.next(n_stages);
        place.next(n_places);
      }
      at.next(a, n_experts);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ draining the sums
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    Place<MODE> at(a, n_experts, u0);
    Turn buf;
    bool begins = true;  // down: the next expert is the first of a tile
    for (int left = n_mine; left > 0; --left) {
      const int slot = at.slot, row = at.row;
      const bool segment_ends = left == 1 || at.kc + 1 == a.k_units;
      const bool tile_ends = left == 1 || at.ends(a, n_experts);
      at.next(a, n_experts);
      if (!segment_ends) continue;
      const int n_row = row * kRows + r;
      const bool in = n_row < a.rows;
      // whose units the tile is made of
      const int tile = MODE == kUp ? slot * a.row_tiles + row : row;
      const int tile_units = a.k_units * (MODE == kDown ? n_experts : 1);
      const long long first = static_cast<long long>(tile) * tile_units;
      const int b0 = owner(first, n_units, ctas), b1 = owner(first + tile_units - 1, n_units, ctas);
      auto part_of = [&](int b) {  // a CTA's tile that began before it is its part 0
        return a.part + (static_cast<size_t>(b) * 2 + (b == b0 ? 1 : 0)) * part_floats(MODE) + r;
      };
      // Whether the tile's other parts are all there, asked while the MMAs still run: those of the CTAs that began with this tile
      // were their first work. The part then stays in registers. (5 tokens of 8 of 128 experts: 85.9 us, by the workspace 87.5.)
      auto others_there = [&]() {
        if (threadIdx.x == 64) {
          unsigned n;
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(a.counters + tile) : "memory");
          const int all = n == static_cast<unsigned>(b1 - b0) && !*abort_flag;
          if (all) a.counters[tile] = 0u;
          __threadfence();
          *there = all;  // once: of the CTA's last tile
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        return *there != 0;
      };
      // after this CTA's part is written: whether all are
      auto last_of_tile = [&]() {
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (threadIdx.x == 64) {
          int is_last = 0;
          if (!*abort_flag) {
            const unsigned before = atomicAdd(a.counters + tile, 1u);
            is_last = before == static_cast<unsigned>(b1 - b0);
            if (is_last) a.counters[tile] = 0u;
          }
          __threadfence();
          *last = is_last;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        return *last != 0;
      };
      const unsigned tokens = MODE == kGemv ? everyone : ex->tokens[slot];
      const int n_tok = __popc(tokens);
      float f = 0.f;  // down: lane's token's weight, times down's factor and h's
      int place = 0;
      if (MODE == kDown && lane < n_tok) {
        place = ex->place[slot][nth_bit(tokens, lane)];
        f = ex->weight[place] * (a.f0 ? __ldg(a.f0 + ex->expert[slot]) : 1.f);
      }
      if (MODE == kDown && begins)
        for (int t = 0; t < a.M; ++t) sums[t * kRows + r] = 0.f;
      begins = tile_ends;
      const bool alone = MODE == kUp && kOwn && left == 1 && b0 != b1 && others_there();
      const bool ok = mbar_wait_warp(smem_u32(&dfull[buf.i]), buf.parity, abort_flag, a.wait_limit, &g_stream_err);
      tc_fence_after();
      // (the largest h is known: parts made with it have come through the MMAs)
      if (MODE == kDown && lane < n_tok)
        f *= pow2(h_exponent(__ldcg(a.h_most + place)) + (FMT == EXQ_FP4_E4M3 ? e4m3_shift(kHTop) : 0));
      float v[kMatrices][kVals];  // the row's values: token by token; up: gate's and up's
#pragma unroll
      for (int w = 0; w < kMatrices; ++w)
#pragma unroll
        for (int j = 0; j < kVals; ++j) v[w][j] = 0.f;
      if (ok) {
        const uint32_t d = tmem + lanes + buf.i * buffer_cols;
#pragma unroll
        for (int j = 0; j < kVals; j += 2) {
          if (j < n_tok) {
            float c[kMatrices][16];
#pragma unroll
            for (int w = 0; w < kMatrices; ++w) tmem_ld16(d + w * cols + 8 * j, c[w]);
#pragma unroll
            for (int w = 0; w < kMatrices; ++w) {
              wait_ld(c[w]);
              v[w][j] = join_parts(c[w]);
              v[w][j + 1] = join_parts(c[w] + 8);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&dempty[buf.i]));
      buf.next(n_buffers);
      if constexpr (MODE == kDown) {
        // an expert's sums go to its own tokens only: a NaN of its weights reaches no other
        unsigned m = tokens;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= n_tok) break;
          const float fj = __shfl_sync(0xffffffffu, f, j);
          const int t = __ffs(static_cast<int>(m)) - 1;
          m &= m - 1u;
          sums[t * kRows + r] = fmaf(v[0][j], fj, sums[t * kRows + r]);
        }
        if (!tile_ends) continue;
#pragma unroll
        for (int t = 0; t < NT; ++t) v[0][t] = t < a.M ? sums[t * kRows + r] : 0.f;
      }

      // ---- the tile, or this CTA's part of it
      const int n_val = MODE == kDown ? a.M : n_tok;
      if (b0 != b1) {
        if (!alone) {
          float* p = part_of(blockIdx.x);
#pragma unroll
          for (int w = 0; w < kMatrices; ++w)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              if (j < n_val) __stcg(p + (w * kMaxTokens + j) * kRows, v[w][j]);
          if (!last_of_tile()) continue;
        }
        add_parts<kOwn>(v, n_val, b0, b1, part_of);
      }
      if constexpr (MODE == kUp) {
        const int id = ex->expert[slot];
        const float fx = FMT == EXQ_FP4_E4M3 ? pow2(e4m3_shift(kXTop)) : 1.f;  // of x's parts
        const float fg = (a.f0 ? __ldg(a.f0 + id) : 1.f) * fx, fu = (a.f1 ? __ldg(a.f1 + id) : 1.f) * fx;
        unsigned m = tokens;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= n_tok) break;
          const int place = ex->place[slot][__ffs(static_cast<int>(m)) - 1];
          m &= m - 1u;
          const float h = activate(v[0][j] * fg, a.act) * (v[kMatrices - 1][j] * fu);
          if (in) a.h[static_cast<size_t>(place) * a.rows + n_row] = h;
          // magnitudes order as their bits do
          const unsigned most = __reduce_max_sync(0xffffffffu, in && isfinite(h) ? __float_as_uint(fabsf(h)) : 0u);
          if (lane == 0) atomicMax(a.h_most + place, most);
        }
      } else if (!*abort_flag && in) {
        const float f = MODE == kGemv ? a.factor * (FMT == EXQ_FP4_E4M3 ? pow2(e4m3_shift(kXTop)) : 1.f) : 1.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (t < a.M) a.y[static_cast<size_t>(t) * a.rows + n_row] = __half_as_ushort(__float2half_rn(v[0][t] * f));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace fp4s
}  // namespace exq
