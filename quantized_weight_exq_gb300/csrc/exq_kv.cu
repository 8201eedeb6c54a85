// Quantized KV cache codec, Q4 / Q6 / Q8.
//
// The ExLlamaV2 blog post ("ExLlamaV2: The fastest inference engine for
// quantized Llama/HF models") lists a Q4 / Q6 / Q8 KV cache (comparison table;
// "Step 2: Use the right cache mode for your context length") and costs it
// at half a byte (Q4) and one byte (Q8) per cached element ("Production
// Considerations", VRAM estimate); the codec itself is not described. This
// one: a group is the D values of one (token, head); symmetric with
// qmax = 2^(b-1) - 1;
//   s = fp16_RN(fp32_RN(amax / qmax)),
//   q = clamp(rint(fp32_RN(x / s)), -qmax - 1, qmax)  (0 where s = 0),
//   u = q + 2^(b-1), code i of the group at bits [i b, i b + b) of its
//   little-endian word stream;
// read back as fp16_RN((u - 2^(b-1)) s). Every integer decision is an IEEE
// fp32 division rounded to nearest even, then round-half-even to an integer.
//
// Both kernels are bound by HBM. A warp handles four groups, lane l holding
// the D / 32 consecutive values [l D/32, (l+1) D/32) of each, so a group moves
// as one contiguous block (D * 2 bytes of fp16, D * b / 8 bytes of codes); all
// of a warp's loads are issued before any of its arithmetic, to keep enough
// bytes in flight per SM.
//
// Below the codec: the append to a paged cache, which runs the same codec on
// rotated keys, and the copy of pages.
#include <algorithm>
#include <type_traits>

#include "exq_device.cuh"
#include "exq_internal.h"
#include "exq_rope.cuh"

namespace exq {
namespace {

constexpr int kWarps = 8;  // groups per 256-thread block

// x / C rounded to nearest even in fp32, for x an fp16 magnitude (amax) and
// C = qmax in {7, 31, 127}: the quotient x y with y = RN(1 / C), corrected by
// one fma with its remainder (the division-by-a-constant method of Cornea,
// Harrison and Tang, "Scientific Computing on Itanium-based Systems", FMA
// correction step). For these C every positive finite fp16 x gives the
// correctly rounded quotient, checked exhaustively against exact rational
// rounding in tests/test_kv_division.py; three instructions instead of a
// full IEEE division.
template <int C>
__device__ __forceinline__ float div_by_const(float x) {
  // RN(1 / C), written out so that it does not depend on constant folding
  constexpr float y = C == 7 ? 0x1.24924ap-3f : C == 31 ? 0x1.084210p-5f : 0x1.020408p-7f;
  const float q = __fmul_rn(x, y);
  const float r = __fmaf_rn(-q, static_cast<float>(C), x);
  return __fmaf_rn(r, y, q);
}

// 1 / s from the hardware's approximate reciprocal (PTX `rcp.approx.ftz.f32`,
// at most 1 ulp from 1 / s over the whole range; s is an fp16 value, so
// never an fp32 subnormal). x * inv is then within |x / s| 2^-22 of
// fp32_RN(x / s): 2^-15 for the codes that are not clamped (|x / s| <=
// 128), half the window below in which the exact quotient decides.
__device__ __forceinline__ float rcp_approx(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

template <int VPL>  // values per lane: D / 32
struct Vec;
template <>
struct Vec<2> {
  using T = uint32_t;
};
template <>
struct Vec<4> {
  using T = uint2;
};
template <>
struct Vec<8> {
  using T = uint4;
};

template <int VPL>
__device__ __forceinline__ void unpack_halves(const typename Vec<VPL>::T& v, uint32_t (&h)[VPL]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) {
    h[2 * i] = w[i] & 0xFFFFu;
    h[2 * i + 1] = w[i] >> 16;
  }
}

constexpr int gcd32(int c) { return c % 32 == 0 ? 32 : c % 16 == 0 ? 16 : c % 8 == 0 ? 8 : 4; }

// The group's code words from the lanes' bit chunks (lane l holds stream bits
// [l C, l C + C), C = kChunk <= 64): word w gathers, by warp shuffles, the at
// most NC chunks that overlap bits [32 w, 32 w + 32). Every lane calls it.
template <int kChunk, int kWords>
__device__ __forceinline__ void store_words(unsigned long long chunk, uint32_t* __restrict__ dst, int lane) {
  if constexpr (kChunk == 64) {  // two whole words per lane
    *reinterpret_cast<uint2*>(dst + 2 * lane) =
        make_uint2(static_cast<uint32_t>(chunk), static_cast<uint32_t>(chunk >> 32));
    return;
  } else if constexpr (kChunk == 32) {  // one whole word per lane
    dst[lane] = static_cast<uint32_t>(chunk);
    return;
  } else if constexpr (kChunk == 24) {  // four lanes fill three words: lane 4k + i (i < 3) writes word 3k + i
    const uint32_t c = static_cast<uint32_t>(chunk);
    const uint32_t next = __shfl_down_sync(0xffffffffu, c, 1);
    const int i = lane & 3;
    if (i < 3) dst[3 * (lane >> 2) + i] = (c >> (8 * i)) | (next << (24 - 8 * i));
    return;
  } else if constexpr (kChunk == 16 || kChunk == 8) {  // 32 / kChunk lanes fill a word
    constexpr int kPer = 32 / kChunk;
    uint32_t word = static_cast<uint32_t>(chunk);
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      word |= __shfl_down_sync(0xffffffffu, static_cast<uint32_t>(chunk), i) << (i * kChunk);
    if (lane % kPer == 0) dst[lane / kPer] = word;
    return;
  }
  constexpr int NC = (kChunk - gcd32(kChunk) + 32 + kChunk - 1) / kChunk;
#pragma unroll
  for (int r = 0; r < (kWords + 31) / 32; ++r) {
    const int w = 32 * r + lane;
    const int l0 = min(32 * w / kChunk, 31);
    const int sh = 32 * w - l0 * kChunk;  // the word's first bit inside chunk l0
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int src = min(l0 + c, 31);
      unsigned long long v;
      if constexpr (kChunk <= 32) {
        v = __shfl_sync(0xffffffffu, static_cast<uint32_t>(chunk), src);
      } else {
        const uint32_t lo = __shfl_sync(0xffffffffu, static_cast<uint32_t>(chunk), src);
        const uint32_t hi = __shfl_sync(0xffffffffu, static_cast<uint32_t>(chunk >> 32), src);
        v = (static_cast<unsigned long long>(hi) << 32) | lo;
      }
      const int pos = c * kChunk - sh;  // chunk l0 + c starts this many bits into the word
      if (l0 + c <= 31 && pos < 32) word |= pos >= 0 ? static_cast<uint32_t>(v << pos) : static_cast<uint32_t>(v >> -pos);
    }
    if (w < kWords) dst[w] = word;
  }
}

// One group from the lanes' values (fp16 bits h): codes and scale.
template <int VPL, int B>
__device__ __forceinline__ void quantize_group(const uint32_t (&h)[VPL], uint32_t* __restrict__ dst,
                                               uint16_t* __restrict__ scale, int lane) {
  constexpr int kWords = VPL * B;      // words of a group: 32 VPL values of B bits
  constexpr int kChunk = VPL * B;      // bits of one lane (8..64)
  constexpr int kQmax = (1 << (B - 1)) - 1;
  float xf[VPL];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    xf[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(h[i])));
    amax = fmaxf(amax, fabsf(xf[i]));
  }
  // non-negative floats order as their bit patterns
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  static_assert(kQmax == 7 || kQmax == 31 || kQmax == 127, "div_by_const is checked for these only");
  const __half s16 = __float2half_rn(div_by_const<kQmax>(amax));
  const float s = __half2float(s16);
  const float inv = s != 0.f ? rcp_approx(s) : 0.f;  // s = 0: every q is 0

  // q = rint(fp32_RN(x / s)): from x * inv, except where that lies within
  // 2^-14 of a half-integer; one test per lane for its VPL values
  int q[VPL];
  bool near_tie = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float r = xf[i] * inv;
    q[i] = __float2int_rn(r);
    near_tie |= fabsf(r - static_cast<float>(q[i])) > 0.5f - 0x1p-14f;
  }
  if (near_tie)
#pragma unroll
    for (int i = 0; i < VPL; ++i) q[i] = __float2int_rn(__fdiv_rn(xf[i], s));
  // A normal fp16 s is within 2^-11 (plus the fp32 quotient's 2^-24) of
  // amax / qmax, so |x / s| < qmax (1 + 2^-10) < qmax + 1/2 and every q is
  // already in range; only a subnormal s (amax < 2^-14 qmax), with fewer
  // significant bits, needs the clamp. The test is the same for the whole
  // warp (s is the group's).
  if (s < 0x1p-14f)
#pragma unroll
    for (int i = 0; i < VPL; ++i) q[i] = max(-kQmax - 1, min(kQmax, q[i]));
  using Chunk = std::conditional_t<(kChunk <= 32), uint32_t, unsigned long long>;
  Chunk chunk = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) chunk |= static_cast<Chunk>(q[i] + (1 << (B - 1))) << (i * B);
  store_words<kChunk, kWords>(chunk, dst, lane);
  if (lane == 0) *scale = __half_as_ushort(s16);
}

template <int VPL, int B, int GPW>
__global__ void __launch_bounds__(kWarps * 32)
    kv_quantize_kernel(const uint16_t* __restrict__ x, long long n_groups, uint32_t* __restrict__ codes,
                       uint16_t* __restrict__ scales) {
  constexpr int D = 32 * VPL;
  constexpr int kWords = D * B / 32;   // words of a group
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the block's groups: k * kWarps + warp, k < GPW (each k a contiguous run of kWarps groups)
  const long long g0 = static_cast<long long>(blockIdx.x) * kWarps * GPW + warp;

  using V = typename Vec<VPL>::T;
  V raw[GPW];
#pragma unroll
  for (int k = 0; k < GPW; ++k) {  // every load of the warp first
    const long long g = g0 + k * kWarps;
    if (g < n_groups) raw[k] = *reinterpret_cast<const V*>(x + g * D + lane * VPL);
  }

#pragma unroll
  for (int k = 0; k < GPW; ++k) {
    const long long g = g0 + k * kWarps;
    if (g >= n_groups) break;  // warp-uniform
    uint32_t h[VPL];
    unpack_halves<VPL>(raw[k], h);
    quantize_group<VPL, B>(h, codes + g * kWords, scales + g, lane);
  }
}

template <int VPL, int B, int GPW>
__global__ void __launch_bounds__(kWarps * 32)
    kv_dequantize_kernel(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scales, long long n_groups,
                         uint16_t* __restrict__ x_out) {
  constexpr int D = 32 * VPL;
  constexpr int kWords = D * B / 32;
  constexpr int kChunk = VPL * B;
  constexpr uint32_t kMask = (1u << B) - 1u;
  constexpr int kZ = 1 << (B - 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long g0 = static_cast<long long>(blockIdx.x) * kWarps * GPW + warp;
  const int off = lane * kChunk;
  constexpr bool kTwo = (kChunk & 31) != 0 || kChunk > 32;  // some lane's bits cross a word boundary

  uint32_t lo[GPW], hi[GPW], sc[GPW];
#pragma unroll
  for (int k = 0; k < GPW; ++k) {  // every load of the warp first
    const long long g = g0 + k * kWarps;
    lo[k] = hi[k] = sc[k] = 0u;
    if (g < n_groups) {
      const uint32_t* gw = codes + g * kWords;
      lo[k] = __ldg(gw + (off >> 5));
      if (kTwo && (off & 31) + kChunk > 32) hi[k] = __ldg(gw + (off >> 5) + 1);  // inside the group
      sc[k] = __ldg(scales + g);
    }
  }
  // (u - z) exactly in fp16: u planted in the mantissa of 1024, then - (1024 + z)
  constexpr uint32_t bias = pack2(f16_bits(-(1024 + kZ)), f16_bits(-(1024 + kZ)));
#pragma unroll
  for (int k = 0; k < GPW; ++k) {
    const long long g = g0 + k * kWarps;
    if (g >= n_groups) break;
    const unsigned long long win = ((static_cast<unsigned long long>(hi[k]) << 32) | lo[k]) >> (off & 31);
    const uint32_t s2 = sc[k] | (sc[k] << 16);
    uint32_t out[VPL / 2];
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) {
      const uint32_t u0 = static_cast<uint32_t>(win >> (2 * i * B)) & kMask;
      const uint32_t u1 = static_cast<uint32_t>(win >> ((2 * i + 1) * B)) & kMask;
      out[i] = hmul2(hadd2(u0 | (u1 << 16) | kMagic, bias), s2);
    }
    using V = typename Vec<VPL>::T;
    *reinterpret_cast<V*>(x_out + g * D + lane * VPL) = *reinterpret_cast<const V*>(out);
  }
}

// ---------------------------------------------------------------- paged cache: append

__device__ unsigned g_kv_err;

struct AppendArgs {
  // batch
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int n_seqs, n_tokens, max_pages, max_q_len, max_kv_len;
  // cache, its arrays at the layer
  uint32_t* codes[2];   // K, V
  uint16_t* scales[2];
  int n_kv_heads, page_size, n_pages;
  // rows
  const uint16_t* in[3];  // q, k, v
  uint16_t* q_out;
  long long ts[4], hs[4]; // strides of q, k, v, q_out
  int n_q;                // query heads (0: none)
  // rotary
  const uint64_t* steps;
  const int32_t* pos;
  double gain;
  int R, interleaved;
  int shift;              // log2 of the tokens of a block
  int rows_per;           // rows (q, k and v heads) of a token that one block does
};

struct TokenPlace {
  int pos;        // rotary position
  int block;      // page, or -1: nothing to do for this token
  int slot;
};

// Where token t goes, by one warp: its sequence is the last with
// q_start <= t (counted by the lanes over all sequences, which also see whether
// q_start falls anywhere: then no token's sequence is certain).
__device__ __forceinline__ TokenPlace find_place(const AppendArgs& a, int t, int lane) {
  int n = 0;
  bool falls = false;
  for (int b = lane; b < a.n_seqs; b += 32) {
    const int start = __ldg(a.q_start + b);
    n += start <= t ? 1 : 0;
    falls |= __ldg(a.q_start + b + 1) < start;
  }
  falls = __any_sync(0xffffffffu, falls);
  const int b = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n))) - 1;
  TokenPlace p{0, -1, 0};
  const int end = __ldg(a.q_start + a.n_seqs);
  if (t >= end && !falls) return p;  // padding
  const int first = b >= 0 ? __ldg(a.q_start + b) : 0, next = b >= 0 ? __ldg(a.q_start + b + 1) : 0;
  bool ok = !falls && b >= 0 && next > t && next - first <= a.max_q_len;  // else q_start is wrong, or a bound
  if (ok) {
    const int len = __ldg(a.kv_len + b), at = len - (next - t);
    ok = len <= a.max_kv_len && at >= 0;  // max_kv_len <= max_pages * page_size
    if (ok) {
      const int page = __ldg(a.page_table + static_cast<long long>(b) * a.max_pages + at / a.page_size);
      ok = page >= 0 && page < a.n_pages;
      if (ok) {
        p.pos = a.pos ? __ldg(a.pos + t) : at;
        p.block = page;
        p.slot = at % a.page_size;
      }
    }
  }
  if (!ok && lane == 0) atomicOr(&g_kv_err, kDevErrBadPage);
  return p;
}

// What a lane needs to turn its values [lane VPL, lane VPL + VPL) of any row
// of a token: y = x c + o s with its partner's value o, products and sum each
// rounded (s is negated for the first of a pair, which is exact, so both
// values of a pair come out as by rope_first and rope_second).
template <int VPL>
struct Turn {
  float c[VPL], s[VPL];
  int from;         // lane that holds the partners of HALF pairs; -1: read them from memory
  bool all, some;   // all / some of the lane's values turn
};

template <int VPL>
__device__ __forceinline__ void load_turn(Turn<VPL>& t, const float2* cs, int R, bool interleaved, int lane) {
  const int half = R / 2, d0 = lane * VPL;
  t.all = d0 + VPL <= R;
  t.some = d0 < R;
  t.from = half % VPL == 0 ? (d0 < half ? lane + half / VPL : lane - half / VPL) & 31 : -1;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int d = d0 + i;
    const bool first = interleaved ? (i & 1) == 0 : d < half;
    const float2 v = d < R ? cs[interleaved ? d / 2 : first ? d : d - half] : make_float2(1.f, 0.f);
    t.c[i] = v.x;
    t.s[i] = first ? -v.y : v.y;
  }
}

// The lane's values turned. Partners of HALF pairs come from the lane that
// holds them (R/2 a multiple of VPL), or from the row in memory.
template <int VPL>
__device__ __forceinline__ void rotate_lane(uint32_t (&h)[VPL], const Turn<VPL>& t, const uint16_t* row, int R,
                                            bool interleaved, int lane) {
  uint32_t other[VPL];
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) other[i] = h[i ^ 1];
  } else if (t.from >= 0) {  // the same for all lanes
#pragma unroll
    for (int i = 0; i < VPL; i += 2) {
      const uint32_t two = __shfl_sync(0xffffffffu, h[i] | (h[i + 1] << 16), t.from);
      other[i] = two & 0xFFFFu;
      other[i + 1] = two >> 16;
    }
  } else {
    const int half = R / 2;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int d = lane * VPL + i;
      other[i] = d < R ? row[d < half ? d + half : d - half] : 0u;
    }
    __syncwarp();  // q_out may be the row itself: every partner is read before any lane writes
  }
  if (!t.some) return;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t y = float_to_half_bits(
        __fadd_rn(__fmul_rn(half_bits_to_float(h[i]), t.c[i]), __fmul_rn(half_bits_to_float(other[i]), t.s[i])));
    h[i] = t.all || lane * VPL + i < R ? y : h[i];
  }
}

// 2 bytes read a value, 2 or B / 8 written. Many tokens (4 sequences of up to
// 2048, 64 + 8 + 8 heads of 128, Q8) take 60 us for 177 MB, 2.9 TB/s: neither
// HBM nor the issue slots (59 %) are full, a warp waits for loads and for the
// steps of a row's codec, maximum, quotient, exchange, one after the other.
// One token takes 7 us, the launch and its dependent steps: a block
// holds 1 .. 8 tokens, each done by 8 / tokens of its warps, and where tokens
// are few the rows of a token are split over blocks. A warp does a row (one
// head of q, k or v) at a time, with the loads of kU rows of each of q, k and
// v in flight before their arithmetic, the first ones while the token's place
// is looked up; cos and sin are computed once per block, and a lane keeps
// those of its values in registers for all rows.
template <int VPL, int B>
__global__ void __launch_bounds__(kWarps * 32, VPL <= 4 ? 3 : 2) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float2 cs[];
  __shared__ TokenPlace places[kWarps];
  constexpr int D = 32 * VPL;
  constexpr int kU = VPL <= 4 ? 4 : 2;
  using V = typename Vec<VPL>::T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = 1 << a.shift;
  const int t0 = blockIdx.x << a.shift;
  const int tk = warp & (tokens - 1), stride = kWarps >> a.shift;
  const long long t = t0 + tk;
  // the block's rows of the token, heads of q, k and v one after the other
  const int begin = blockIdx.y * a.rows_per, end = begin + a.rows_per;

  // heads [first, last) of q, k or v, every `stride`-th from the warp's own
  struct Part {
    int first, last;
    const uint16_t* src;  // of head `first`
    long long step;
  };
  const auto part_of = [&](int which, int start, int heads) {
    Part p;
    int r = begin + (warp >> a.shift);  // the warp's rows are begin + warp / tokens + i stride
    if (r < start) r += (start - r + stride - 1) / stride * stride;
    p.first = r - start;
    p.last = t < a.n_tokens ? min(heads, end - start) : 0;
    p.src = a.in[which] + t * a.ts[which] + p.first * a.hs[which] + lane * VPL;  // (not read where there are no rows)
    p.step = stride * a.hs[which];
    return p;
  };
  const auto fetch = [&](V (&v)[kU], const Part& p, int head, const uint16_t* src) {
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (head + k * stride < p.last) v[k] = *reinterpret_cast<const V*>(src + k * p.step);
  };
  const Part pk = part_of(1, a.n_q, a.n_kv_heads), pv = part_of(2, a.n_q + a.n_kv_heads, a.n_kv_heads);
  const Part pq = part_of(0, 0, a.n_q);
  V vk[kU], vv[kU], next[kU];
  fetch(vk, pk, pk.first, pk.src);
  fetch(vv, pv, pv.first, pv.src);
  fetch(next, pq, pq.first, pq.src);

  if (warp < tokens) {
    TokenPlace p{0, -1, 0};
    if (t0 + warp < a.n_tokens) p = find_place(a, t0 + warp, lane);
    if (lane == 0) places[warp] = p;
  }
  __syncthreads();
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < tokens * half; i += kWarps * 32) {  // R = 0: no rotary positions
    const int of = i / half, j = i - of * half;
    if (places[of].block >= 0)
      cs[i] = rope_cos_sin(__ldg(reinterpret_cast<const unsigned long long*>(a.steps) + j), places[of].pos, a.gain, false);
  }
  __syncthreads();
  const TokenPlace place = places[tk];
  if (place.block < 0) return;  // warp-uniform
  Turn<VPL> turn;
  if (half > 0) load_turn<VPL>(turn, cs + tk * half, a.R, a.interleaved, lane);

  const auto store16 = [&](uint16_t* dst, const uint32_t (&h)[VPL]) {
    uint32_t out[VPL / 2];
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) out[i] = h[2 * i] | (h[2 * i + 1] << 16);
    *reinterpret_cast<V*>(dst + lane * VPL) = *reinterpret_cast<const V*>(out);
  };
  // K (turned) and V to the page
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const Part& p = which ? pv : pk;
    V (&v)[kU] = which ? vv : vk;
    const uint16_t* src = p.src;
    for (int head = p.first; head < p.last; head += kU * stride, src += kU * p.step) {
      if (head != p.first) fetch(v, p, head, src);
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const int hd = head + k * stride;
        if (hd >= p.last) break;  // warp-uniform
        uint32_t h[VPL];
        unpack_halves<VPL>(v[k], h);
        if (which == 0 && half > 0) rotate_lane<VPL>(h, turn, src + k * p.step - lane * VPL, a.R, a.interleaved, lane);
        const long long g = (static_cast<long long>(place.block) * a.n_kv_heads + hd) * a.page_size + place.slot;
        if constexpr (B == 16)
          store16(reinterpret_cast<uint16_t*>(a.codes[which]) + g * D, h);
        else
          quantize_group<VPL, B>(h, a.codes[which] + g * (VPL * B), a.scales[which] + g, lane);
      }
    }
  }
  // Q
  if (a.n_q == 0) return;
  const uint16_t* src = pq.src;
  uint16_t* dst = a.q_out + t * a.ts[3] + pq.first * a.hs[3];
  for (int head = pq.first; head < pq.last; head += kU * stride) {
    V v[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) v[k] = next[k];
    const uint16_t* at = src;
    src += kU * pq.step;
    fetch(next, pq, head + kU * stride, src);
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (head + k * stride >= pq.last) break;  // warp-uniform
      uint32_t h[VPL];
      unpack_halves<VPL>(v[k], h);
      rotate_lane<VPL>(h, turn, at + k * pq.step - lane * VPL, a.R, a.interleaved, lane);
      store16(dst, h);
      dst += stride * a.hs[3];
    }
  }
}

// ---------------------------------------------------------------- paged cache: copies

struct CopyArgs {
  uint8_t* base[4];          // k_codes, v_codes, k_scales, v_scales
  long long page_bytes[4];   // 0: absent
  int pieces[4];             // pieces of kCopyPiece bytes of a page of each
  int per_page;              // their sum
  const int32_t* pairs;
  long long n_pairs;
  int n_pages, n_layers;
};

constexpr int kCopyPiece = 256 * 16 * 4;  // four 16-byte loads in flight a thread

// Bound by HBM (1500 pages in 8 layers, 6.3 GB: 997 us, 94 % of the copy
// rate): a block takes pieces of 16 KB, of any (pair, layer, array) in
// turn, and issues a piece's loads before its stores.
__global__ void __launch_bounds__(256) kv_copy_kernel(const __grid_constant__ CopyArgs a) {
  const long long total = a.n_pairs * a.n_layers * a.per_page;
  for (long long w = blockIdx.x; w < total; w += gridDim.x) {
    const long long pl = w / a.per_page;
    int piece = static_cast<int>(w - pl * a.per_page);
    const int layer = static_cast<int>(pl % a.n_layers);
    const long long pair = pl / a.n_layers;
    const int src = __ldg(a.pairs + 2 * pair), dst = __ldg(a.pairs + 2 * pair + 1);
    if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages) {
      if (threadIdx.x == 0) atomicOr(&g_kv_err, kDevErrBadPage);
      continue;
    }
    int k = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (k == i && piece >= a.pieces[i]) {
        piece -= a.pieces[i];
        k = i + 1;
      }
    const long long bytes = k == 0 ? a.page_bytes[0] : k == 1 ? a.page_bytes[1] : k == 2 ? a.page_bytes[2] : a.page_bytes[3];
    uint8_t* base = k == 0 ? a.base[0] : k == 1 ? a.base[1] : k == 2 ? a.base[2] : a.base[3];
    const long long layer0 = static_cast<long long>(layer) * a.n_pages;
    const uint4* from = reinterpret_cast<const uint4*>(base + (layer0 + src) * bytes);
    uint4* to = reinterpret_cast<uint4*>(base + (layer0 + dst) * bytes);
    const long long i0 = static_cast<long long>(piece) * (kCopyPiece / 16) + threadIdx.x, n = bytes / 16;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + 256 * j < n) v[j] = __ldcs(from + i0 + 256 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + 256 * j < n) __stcs(to + i0 + 256 * j, v[j]);
  }
}

// ---------------------------------------------------------------- launches

constexpr int kGpw = 4;  // groups per warp

using QuantFn = void (*)(const uint16_t*, long long, uint32_t*, uint16_t*);
using DequantFn = void (*)(const uint32_t*, const uint16_t*, long long, uint16_t*);

template <int VPL>
QuantFn quant_for_bits(int b) {
  return b == 4 ? kv_quantize_kernel<VPL, 4, kGpw>
                : b == 6 ? kv_quantize_kernel<VPL, 6, kGpw> : kv_quantize_kernel<VPL, 8, kGpw>;
}
template <int VPL>
DequantFn dequant_for_bits(int b) {
  return b == 4 ? kv_dequantize_kernel<VPL, 4, kGpw>
                : b == 6 ? kv_dequantize_kernel<VPL, 6, kGpw> : kv_dequantize_kernel<VPL, 8, kGpw>;
}

dim3 grid_for(long long n_groups) {
  return dim3(static_cast<unsigned>((n_groups + kWarps * kGpw - 1) / (kWarps * kGpw)));
}

}  // namespace

exq_status launch_kv_quantize(const uint16_t* x, long long n_groups, int D, int b, uint32_t* codes,
                              uint16_t* scales, cudaStream_t stream) {
  if (n_groups == 0) return EXQ_OK;
  const QuantFn fn = D == 64 ? quant_for_bits<2>(b) : D == 128 ? quant_for_bits<4>(b) : quant_for_bits<8>(b);
  fn<<<grid_for(n_groups), kWarps * 32, 0, stream>>>(x, n_groups, codes, scales);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

exq_status launch_kv_dequantize(const uint32_t* codes, const uint16_t* scales, long long n_groups, int D, int b,
                                uint16_t* x_out, cudaStream_t stream) {
  if (n_groups == 0) return EXQ_OK;
  const DequantFn fn =
      D == 64 ? dequant_for_bits<2>(b) : D == 128 ? dequant_for_bits<4>(b) : dequant_for_bits<8>(b);
  fn<<<grid_for(n_groups), kWarps * 32, 0, stream>>>(codes, scales, n_groups, x_out);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

namespace {

template <int VPL>
void (*append_for_bits(int b))(const AppendArgs) {
  return b == 4 ? kv_append_kernel<VPL, 4>
                : b == 6 ? kv_append_kernel<VPL, 6> : b == 8 ? kv_append_kernel<VPL, 8> : kv_append_kernel<VPL, 16>;
}

}  // namespace

exq_status launch_kv_append(const exq_kv_cache& c, int layer, const exq_kv_batch& batch, const exq_rows& k,
                            const exq_rows& v, const exq_rope_params* rope, const int32_t* pos, const exq_rows* q,
                            const exq_rows* q_out, int n_heads, int sms, cudaStream_t stream) {
  AppendArgs a{};
  a.q_start = batch.q_start;
  a.kv_len = batch.kv_len;
  a.page_table = batch.page_table;
  a.n_seqs = batch.n_seqs;
  a.n_tokens = batch.n_tokens;
  a.max_pages = batch.max_pages;
  a.max_q_len = batch.max_q_len;
  a.max_kv_len = batch.max_kv_len;
  const long long groups = static_cast<long long>(c.n_pages) * c.n_kv_heads * c.page_size * layer;  // before the layer
  a.codes[0] = c.k_codes + groups * (c.D * c.bits / 32);
  a.codes[1] = c.v_codes + groups * (c.D * c.bits / 32);
  if (c.bits != 16) {
    a.scales[0] = c.k_scales + groups;
    a.scales[1] = c.v_scales + groups;
  }
  a.n_kv_heads = c.n_kv_heads;
  a.page_size = c.page_size;
  a.n_pages = c.n_pages;
  const exq_rows* rows[3] = {q, &k, &v};
  for (int i = 0; i < 3; ++i)
    if (rows[i]) {
      a.in[i] = rows[i]->data;
      a.ts[i] = rows[i]->token_stride;
      a.hs[i] = rows[i]->head_stride;
    }
  if (q) {
    a.q_out = q_out->data;
    a.ts[3] = q_out->token_stride;
    a.hs[3] = q_out->head_stride;
    a.n_q = n_heads;
  }
  if (rope) {
    a.steps = rope->steps;
    a.pos = pos;
    a.gain = rope->gain;
    a.R = rope->R;
    a.interleaved = rope->layout == EXQ_ROPE_INTERLEAVED;
  }
  // tokens of a block: about one cos and sin a thread, and enough blocks to fill the SMs
  const int all = a.n_q + 2 * a.n_kv_heads;
  while (a.shift < 3 && (a.R / 2) << (a.shift + 1) <= kWarps * 32 && (a.n_tokens >> (a.shift + 1)) >= 2 * sms) ++a.shift;
  const int gx = static_cast<int>((static_cast<long long>(a.n_tokens) + (1 << a.shift) - 1) >> a.shift);
  const int splits = std::min(std::max(1, (2 * sms + gx - 1) / gx), (all + kWarps - 1) / kWarps);
  a.rows_per = (all + splits - 1) / splits;
  const dim3 grid(gx, (all + a.rows_per - 1) / a.rows_per);
  const size_t smem = (static_cast<size_t>(a.R / 2) << a.shift) * sizeof(float2);
  auto fn = c.D == 64 ? append_for_bits<2>(c.bits) : c.D == 128 ? append_for_bits<4>(c.bits) : append_for_bits<8>(c.bits);
  fn<<<grid, kWarps * 32, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

exq_status launch_kv_copy(const exq_kv_cache& c, const int32_t* pairs, long long n_pairs, int sms, cudaStream_t stream) {
  CopyArgs a{};
  const long long slots = static_cast<long long>(c.n_kv_heads) * c.page_size;
  void* base[4] = {c.k_codes, c.v_codes, c.k_scales, c.v_scales};
  for (int i = 0; i < 4; ++i) {
    a.base[i] = static_cast<uint8_t*>(base[i]);
    a.page_bytes[i] = i < 2 ? slots * c.D * c.bits / 8 : c.bits == 16 ? 0 : slots * 2;
    a.pieces[i] = static_cast<int>((a.page_bytes[i] + kCopyPiece - 1) / kCopyPiece);
    a.per_page += a.pieces[i];
  }
  a.pairs = pairs;
  a.n_pairs = n_pairs;
  a.n_pages = c.n_pages;
  a.n_layers = c.n_layers;
  const long long total = n_pairs * c.n_layers * a.per_page;
  kv_copy_kernel<<<static_cast<unsigned>(std::min<long long>(total, 8ll * sms)), 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

unsigned take_kv_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_kv_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_kv_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
