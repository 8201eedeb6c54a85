// What the paged attention kernels share: their arguments, the division of
// the work over CTAs, the join of split units, and PTX wrappers.
//
// Work is cut into units: a block of query rows of one sequence and KV head
// (row r of a sequence and KV head is new token r / group, query head
// r % group of it, so the rows of one token lie together), over the tiles of
// cached tokens that some row of the block sees. What a unit costs beside its
// tiles (loading its queries, bringing its sums together) counts as
// `unit_cost` tiles before its first. All units, one after the other, are
// divided evenly over the CTAs, whatever the sequences' lengths: a CTA may end
// a unit that another began, do several whole units, and begin another.
// Lengths are read on the device. A unit that several CTAs share is joined by
// the last of them to finish, in the CTAs' order, so the result does not
// depend on which one that is.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "exq_device.cuh"
#include "exq_internal.h"
#include "exq_rope.cuh"

namespace exq {

struct AttnArgs {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int n_seqs, n_tokens, max_pages, max_q_len, max_kv_len;
  const uint32_t* codes[2];   // K, V of the layer
  const uint16_t* scales[2];
  int n_kv_heads, page_size, n_pages, group;  // group: query heads of a KV head
  exq_rows q, out;
  int n_heads;
  float scale_log2;           // scale * log2(e)
  int causal, window;
  float* lse;
  int rows_above, rows_upto;  // the launch serves sequences of rows_above < rows <= rows_upto a KV head
  int row_blocks;             // blocks of rows such a sequence may need (host bound)
  int unit_cost;              // what a unit costs beside its tiles, in tiles
  int min_tiles;              // fewest tiles worth a CTA
  unsigned* counters;         // [CTAs], zero between calls
  float* partial;             // [CTAs][2][rows * (D + 2)]
  unsigned* err;              // the device error word
  int wait_limit;
  int starve;
};

constexpr size_t kAttnCounterBytes = 64 << 10;
constexpr int kAttnMaxCtas = static_cast<int>(kAttnCounterBytes / sizeof(unsigned));

// Geometry of a block of rows: sequence b, its new tokens and lengths, the
// rows, and the tiles [tile0, tile0 + tiles) of cached tokens [begin, end).
struct AttnUnit {
  int b, q0, n, len;   // sequence, its first row of q, new tokens, cached tokens
  int r0, rows;        // first row of the block, rows of it
  int begin, end;      // cached tokens that some row sees
  int tile0, tiles;    // tiles >= 1 where rows > 0 (one, empty, where nothing is seen)
};

template <int ROWS, int TILE>
__device__ __forceinline__ AttnUnit attn_unit(const AttnArgs& a, int pair) {
  AttnUnit u{};
  u.b = a.row_blocks == 1 ? pair : pair / a.row_blocks;
  const int rb = a.row_blocks == 1 ? 0 : pair - u.b * a.row_blocks;
  u.q0 = __ldg(a.q_start + u.b);
  u.n = __ldg(a.q_start + u.b + 1) - u.q0;
  u.len = __ldg(a.kv_len + u.b);
  if (u.q0 < 0 || u.n < 0 || u.n > a.max_q_len || u.q0 > a.n_tokens - u.n || u.len < 0 || u.len > a.max_kv_len) {
    atomicOr(a.err, kDevErrBadPage);
    return u;
  }
  const int all = u.n * a.group;
  u.r0 = rb * ROWS;
  u.rows = all > a.rows_above && all <= a.rows_upto ? min(ROWS, all - u.r0) : 0;
  if (u.rows <= 0) {
    u.rows = 0;
    return u;
  }
  const int first = u.len - u.n + u.r0 / a.group, last = u.len - u.n + (u.r0 + u.rows - 1) / a.group;  // positions
  u.end = a.causal ? min(u.len, max(0, last + 1)) : u.len;
  u.begin = a.window > 0 ? max(0, first - a.window + 1) : 0;
  if (u.begin >= u.end) {
    u.begin = u.end = u.tile0 = 0;
    u.tiles = 1;
  } else {
    u.tile0 = u.begin / TILE;
    u.tiles = (u.end + TILE - 1) / TILE - u.tile0;
  }
  return u;
}

// The pair after one whose unit is u. Blocks past a sequence's rows are passed
// over together: one prompt chunk among many single tokens gives every
// sequence as many blocks as the chunk.
__device__ __forceinline__ int attn_after(const AttnArgs& a, int pair, const AttnUnit& u) {
  return u.rows > 0 ? pair + 1 : (u.b + 1) * a.row_blocks;
}

// Places of a unit in the division.
__device__ __forceinline__ long long attn_places(const AttnArgs& a, const AttnUnit& u) {
  return u.tiles > 0 ? u.tiles + a.unit_cost : 0;
}

// A CTA's share of the places: [begin, end) of `total`, and where it starts.
// The first `extra` CTAs have per + 1 places, the others per.
struct AttnShare {
  long long total, begin, end;
  long long pair_start;  // places before the first pair, all heads
  long long per;
  int extra;
  int pair;
  int ctas;              // CTAs that have work
};

// quotients of non-negative numbers, by the short division where it does
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Every warp works it out for itself, each lane for its part of the pairs:
// no shared memory, no barrier.
template <int ROWS, int TILE>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& a) {
  const int lane = threadIdx.x & 31;
  const int pairs = a.n_seqs * a.row_blocks;
  const int per = (pairs + 31) >> 5, p0 = min(lane * per, pairs), p1 = min(p0 + per, pairs);
  long long sum = 0;
  for (int p = p0; p < p1;) {
    const AttnUnit u = attn_unit<ROWS, TILE>(a, p);
    sum += attn_places(a, u);
    p = attn_after(a, p, u);
  }
  long long inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += v;
  }
  AttnShare s;
  s.total = __shfl_sync(0xffffffffu, inc, 31) * a.n_kv_heads;
  s.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), quotient(s.total + a.min_tiles - 1, a.min_tiles)));
  s.begin = s.end = s.pair_start = s.per = 0;
  s.pair = s.extra = 0;
  const int cta = blockIdx.x;
  if (cta >= s.ctas) return s;
  s.per = quotient(s.total, s.ctas);
  s.extra = static_cast<int>(s.total - s.per * s.ctas);
  s.begin = cta * s.per + min(cta, s.extra);
  s.end = s.begin + s.per + (cta < s.extra ? 1 : 0);
  long long at = (inc - sum) * a.n_kv_heads;  // places before this lane's pairs
  const bool mine = at <= s.begin && s.begin < at + sum * a.n_kv_heads;
  int pair = p0;
  if (mine && per > 1)
    while (pair < p1 - 1) {
      const AttnUnit u = attn_unit<ROWS, TILE>(a, pair);
      const long long places = attn_places(a, u) * a.n_kv_heads;
      if (s.begin < at + places) break;
      at += places;
      pair = attn_after(a, pair, u);
    }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;  // one lane
  s.pair_start = __shfl_sync(0xffffffffu, at, from);
  s.pair = __shfl_sync(0xffffffffu, pair, from);
  return s;
}

// The CTA whose share holds place x.
__device__ __forceinline__ int attn_cta_of(const AttnShare& s, long long x) {
  const long long longer = s.extra * (s.per + 1);  // places of the CTAs that have one more
  return static_cast<int>(x < longer ? quotient(x, s.per + 1) : s.extra + quotient(x - longer, s.per));
}

// A CTA's piece of a unit, in order.
struct AttnPiece {
  AttnUnit u;
  int head;            // KV head
  int t0, t1;          // tiles of the piece, counted from cached token 0
  long long first;     // the place of the unit's first tile
  bool whole;
};

// A warp's place in its CTA's share and the piece it is at. It lies in shared
// memory, one for each warp (all of a CTA's warps go through the same pieces):
// in registers it would be carried, and spilled, through the loops over tiles.
struct AttnState {
  AttnShare s;
  long long at;          // next place of the share
  long long pair_start;
  int pair;
  int number;            // of the piece, from 1
  AttnPiece p;
};

template <int ROWS, int TILE>
__device__ __forceinline__ bool attn_begin(const AttnArgs& a, AttnState& st) {
  const AttnShare s = attn_share<ROWS, TILE>(a);
  if ((threadIdx.x & 31) == 0) {
    st.s = s;
    st.at = s.begin;
    st.number = 0;
    st.pair = s.pair;
    st.pair_start = s.pair_start;
  }
  __syncwarp();
  return s.begin < s.end;
}

// The next piece, to st.p; false when there is none. Called by whole warps.
template <int ROWS, int TILE>
__device__ __forceinline__ bool attn_next(const AttnArgs& a, AttnState& st) {
  long long at = st.at, pair_start = st.pair_start;
  const long long end = st.s.end;
  int pair = st.pair;
  AttnPiece p;
  for (;;) {
    if (at >= end) return false;  // the same for all lanes
    p.u = attn_unit<ROWS, TILE>(a, pair);
    int places = static_cast<int>(attn_places(a, p.u));
    while (at >= pair_start + static_cast<long long>(places) * a.n_kv_heads) {  // pairs that are done or have no rows
      pair_start += static_cast<long long>(places) * a.n_kv_heads;
      pair = attn_after(a, pair, p.u);
      p.u = attn_unit<ROWS, TILE>(a, pair);
      places = static_cast<int>(attn_places(a, p.u));
    }
    const int off = static_cast<int>(at - pair_start);
    p.head = off / places;
    const int o = off - p.head * places;  // the share's first place in the unit
    const int n = static_cast<int>(min(end - at, static_cast<long long>(places - o)));
    const int from = max(o - a.unit_cost, 0), to = max(o + n - a.unit_cost, 0);
    p.first = at - o + a.unit_cost;
    p.t0 = p.u.tile0 + from;
    p.t1 = p.u.tile0 + to;
    p.whole = to - from == p.u.tiles;
    at += n;
    if (to > from) break;  // else only the unit's cost fell to this CTA
  }
  __syncwarp();  // every lane has read the state
  if ((threadIdx.x & 31) == 0) {
    st.at = at;
    st.pair = pair;
    st.pair_start = pair_start;
    ++st.number;
    st.p = p;
  }
  __syncwarp();
  return true;
}

// The partial result of CTA c in a unit: its second slot where the unit
// begins in the CTA's share, its first where it began before. Row-major
// [rows][D] sums, then [rows] maxima (log2) and [rows] sums of weights.
__device__ __forceinline__ float* attn_slot(const AttnArgs& a, int cta, bool begins, int floats) {
  return a.partial + (static_cast<size_t>(cta) * 2 + (begins ? 1 : 0)) * floats;
}

__device__ __forceinline__ void attn_row_of(const AttnArgs& a, const AttnPiece& p, int r, int& token, int& head) {
  const int rr = p.u.r0 + r;
  const int t = rr / a.group;
  token = p.u.q0 + t;
  head = p.head * a.group + (rr - t * a.group);
}

__device__ __forceinline__ bool attn_finite(uint32_t half_bits) { return (half_bits & 0x7C00u) != 0x7C00u; }

// A K scale as it multiplies its group's products. An infinite one gives NaN,
// as its values do: those of zero codes are NaN, the others infinities of both
// signs.
__device__ __forceinline__ float attn_key_scale(uint32_t half_bits) {
  const float s = half_bits_to_float(half_bits);
  return fmaf(s, 0.f, s);
}

// ---- values that are not finite, at positions that only some rows see
//
// A weight of 0 does not keep an infinity or a NaN of V out of a product. A V
// scale that is not finite is therefore taken as 0 and its token's scores as
// NaN: rows that see the token are NaN, and no others. (Leaving it out where
// the weight is 0 instead would keep the log-sum-exp finite: 893 us for 882 of
// a prompt chunk Q4, 926 for 900 Q8.) fp16 pages go into the matrix product as they are, so their
// tiles with tokens that not every row of the unit sees are cleaned: such a
// token's values are taken as zeros where they are not finite, tokens that no
// row sees as zeros altogether. What was taken out marks the unit, and is
// added again to the rows that do see it when they have been stored, from the
// cache. (The weight of a seen token counts as above 0 there, also where its
// exponential is not: infinity times it is infinity.)

// The cached tokens that every row of the unit sees.
struct AttnSpan {
  int lo, hi;
};
__device__ __forceinline__ AttnSpan attn_seen_by_all(const AttnArgs& a, const AttnUnit& u) {
  const int first = u.len - u.n + u.r0 / a.group, last = u.len - u.n + (u.r0 + u.rows - 1) / a.group;  // positions
  return {a.window > 0 ? max(0, last - a.window + 1) : 0, a.causal ? min(u.len, max(0, first + 1)) : u.len};
}

// the halves of two fp16 values that are not finite, and of those that `among` has the top bit of, as a mask
__device__ __forceinline__ uint32_t attn_not_finite(uint32_t two, uint32_t among) {
  const uint32_t t = ((two & 0x7C007C00u) + 0x04000400u) & 0x80008000u & among;
  return (t >> 15) * 0xFFFFu;
}

// What the cleaning took out of dims [d, d + 4) of fp16 V for row r of the piece: the sum of the values that are not finite,
// of the tokens that row r sees and not every row does. 0: nothing.
template <int D>
__device__ __forceinline__ float4 attn_taken_out(const AttnArgs& a, const AttnPiece& p, int tile, int r, int d) {
  const AttnSpan all = attn_seen_by_all(a, p.u);
  const int pos = p.u.len - p.u.n + (p.u.r0 + r) / a.group;
  const int lo = max(p.t0 * tile, a.window > 0 ? max(0, pos - a.window + 1) : 0);
  const int hi = min(p.t1 * tile, a.causal ? min(p.u.len, pos + 1) : p.u.len);
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int t = lo; t < hi; ++t) {
    if (t >= all.lo && t < all.hi) t = all.hi;
    if (t >= hi) break;
    const int page = __ldg(a.page_table + static_cast<long long>(p.u.b) * a.max_pages + t / a.page_size);
    if (page < 0 || page >= a.n_pages) continue;
    const long long g = (static_cast<long long>(page) * a.n_kv_heads + p.head) * a.page_size + t % a.page_size;
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.codes[1] + (g * D + d) / 2));
    const uint32_t h[4] = {v.x & 0xFFFFu, v.x >> 16, v.y & 0xFFFFu, v.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!attn_finite(h[i])) y[i] += half_bits_to_float(h[i]);
  }
  return make_float4(y[0], y[1], y[2], y[3]);
}

// Adds it to a stored row: fp16 results (`out`), or a piece's fp32 sums (`slot`, not NULL).
template <int D>
__device__ __forceinline__ void attn_put_back(const AttnArgs& a, const AttnPiece& p, int tile, int r, int d, uint16_t* out,
                                              float* slot) {
  const float4 z = attn_taken_out<D>(a, p, tile, r, d);
  const float add[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (add[i] == 0.f) continue;
    if (slot)
      slot[d + i] += add[i];
    else
      out[d + i] = static_cast<uint16_t>(float_to_half_bits(half_bits_to_float(out[d + i]) + add[i]));
  }
}

// References of the softmax. Weights are multiplied by V's scales and rounded
// to fp16 for the matrix instructions: the one rounding to fewer than 32 bits
// before the result's own. (Results are 2.4e-4 to 3.1e-4 of their size off the
// 64-bit ones, 2.1e-4 with their own rounding alone; a second product with the
// remainders would take the matrix instructions of P V twice.) What has to stay
// in fp16's normal range is that product: a row's reference is the largest score plus the
// exponent of its token's V scale (0 for fp16 pages), over the tokens that the
// row sees, and is raised where one exceeds it by more than attn_lag. Weights
// up to 2^lag have the same relative precision; those whose product falls
// below 2^-14 lose some, 2^-25 of the row's largest product at most each. Most
// tiles need no maximum over lanes: one vote, on the lane's largest score plus
// the largest exponent of all its tokens, says that no reference moves.
// (Reference and exponent apart, with the exponent of the largest V scale met,
// let a large scale that a row does not see, or hardly weighs, push the row's
// other products below fp16's range.)
template <int B>
__device__ __forceinline__ constexpr float attn_lag() {
  return B == 16 ? 8.f : 12.f;
}

// The exponent of a V scale (an fp16 value): 2^e <= |v| < 2^(e + 1), -24 (fp16's
// least) for 0; planted in the mantissa of 2^23 rather than converted.
__device__ __forceinline__ float attn_value_exponent(float v) {
  return fmaxf(-24.f, __uint_as_float(0x4B000000u | ((__float_as_uint(v) >> 23) & 255u)) - (8388608.f + 127.f));
}

// A sum of weights of 0 is that of a row that has seen nothing (yet). A NaN
// score makes it NaN, which every step keeps: tests of it are `l != 0`, true
// for NaN.
__device__ __forceinline__ void attn_store_lse(const AttnArgs& a, int token, int head, float m, float l) {
  if (a.lse)
    a.lse[static_cast<long long>(token) * a.n_heads + head] =
        l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

__device__ __forceinline__ float exp2_fast(float x) {  // ex2.approx: 2 ulp, 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Joins the pieces of a unit that CTAs c0 .. c1 share, in their order, and
// writes its rows, in the one CTA that came last. `threads` threads with ids
// `tid` call it. The loads of 8 pieces are in flight at a time, for two
// places (a row, 4 columns) a thread.
template <int ROWS, int D>
__device__ __forceinline__ void attn_join(const AttnArgs& a, const AttnPiece& p, int c0, int c1, int tid, int threads) {
  constexpr int kFloats = ROWS * (D + 2);
  constexpr int kCols = D / 4;
  constexpr int kKeep = 2, kBatch = 8;
  const int places = p.u.rows * kCols;
  for (int e0 = tid; e0 < places; e0 += kKeep * threads) {
    float4 y[kKeep];
    float l[kKeep], m[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f), l[k] = 0.f, m[k] = -INFINITY;
    for (int b0 = c0; b0 <= c1; b0 += kBatch) {
      float4 v[kKeep][kBatch];
      float mi[kKeep][kBatch], li[kKeep][kBatch];
#pragma unroll
      for (int k = 0; k < kKeep; ++k) {
        const int e = min(e0 + k * threads, places - 1), r = e / kCols, col = e - r * kCols;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int c = min(b0 + i, c1);
          const float* s = attn_slot(a, c, c == c0, kFloats);
          v[k][i] = __ldcg(reinterpret_cast<const float4*>(s + r * D) + col);
          mi[k][i] = __ldcg(s + ROWS * D + r);
          li[k][i] = b0 + i <= c1 ? __ldcg(s + ROWS * D + ROWS + r) : 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < kKeep; ++k) {
        float top = m[k];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = li[k][i] != 0.f ? fmaxf(top, mi[k][i]) : top;
        const float old = m[k] == -INFINITY ? 0.f : exp2_fast(m[k] - top);
        l[k] *= old;
        y[k].x *= old, y[k].y *= old, y[k].z *= old, y[k].w *= old;
        m[k] = top;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float f = li[k][i] != 0.f ? exp2_fast(mi[k][i] - top) : 0.f;
          l[k] += li[k][i] * f;
          if (f != 0.f) {
            y[k].x += v[k][i].x * f;
            y[k].y += v[k][i].y * f;
            y[k].z += v[k][i].z * f;
            y[k].w += v[k][i].w * f;
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int e = e0 + k * threads;
      if (e >= places) break;
      const int r = e / kCols, col = e - r * kCols;
      int token, head;
      attn_row_of(a, p, r, token, head);
      const float inv = l[k] != 0.f ? 1.f / l[k] : 0.f;
      uint2 o;
      o.x = float_to_half_bits(y[k].x * inv) | (float_to_half_bits(y[k].y * inv) << 16);
      o.y = float_to_half_bits(y[k].z * inv) | (float_to_half_bits(y[k].w * inv) << 16);
      *reinterpret_cast<uint2*>(a.out.data + token * a.out.token_stride + head * a.out.head_stride + 4 * col) = o;
      if (col == 0) attn_store_lse(a, token, head, m[k], l[k]);
    }
  }
}

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a whole warp, all lanes leave in the same round; false (and a
// recorded timeout) if the phase never completes, or if another role of the
// CTA gave up.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, const AttnArgs& a) {
  for (int i = 0; i < a.wait_limit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
  }
  if ((threadIdx.x & 31) == 0) atomicOr(a.err, kDevErrTimeout);
  *abort_flag = 1;
  return false;
}

}  // namespace exq
