// Rotary positions of rows in memory (exq_rope): y1 = x1 c - x2 s,
// y2 = x2 c + x1 s over the pairs of the first R values of each head.
//
// Bound by HBM: 2 bytes in and 2 out per value. A block takes kTokens tokens
// (as many as give each thread about one pair of cos and sin to compute) and
// all or a part of the heads. cos and sin go to shared memory once; then a
// thread keeps the same 8 pairs (one or two 16-byte chunks of the head) and
// walks over heads, four at a time, their loads issued before the arithmetic.
// 8000 tokens x 64 heads of 128 (262 MB): 53 us, 5.0 TB/s, 74 % of the copy
// rate; the wait for the table at each block's beginning is the rest.
#include <algorithm>

#include "exq_internal.h"
#include "exq_rope.cuh"

namespace exq {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  const uint64_t* steps;
  const int32_t* pos;
  const uint16_t* x;
  uint16_t* y;
  long long xt, xh, yt, yh;  // strides, in values
  long long n_tokens;
  int n_heads, D, R;
  int heads_per;             // heads of one block (grid.y splits them)
  int tokens_per;            // tokens of one block
  int units;                 // thread's places in a head (see the kernels)
  double gain;
  int grad;
};

__device__ __forceinline__ void fill_table(const RopeArgs& a, float2* cs, long long t0, int tokens) {
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int tk = i / half, j = i - tk * half;
    cs[i] = rope_cos_sin(__ldg(reinterpret_cast<const unsigned long long*>(a.steps) + j), __ldg(a.pos + t0 + tk), a.gain,
                         a.grad != 0);
  }
  __syncthreads();
}

// A place in a head is 8 pairs: the chunks of 8 values u and u + R/16 (HALF,
// R % 16 == 0), or the two chunks' worth 2u, 2u + 1 of neighbours
// (INTERLEAVED: one chunk of 8 values holds 4 pairs; R % 8 == 0); places past
// those are chunks that pass through.
template <bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens_per;
  const int tokens = static_cast<int>(min(static_cast<long long>(a.tokens_per), a.n_tokens - t0));
  fill_table(a, cs, t0, tokens);

  const int lanes = a.units * a.tokens_per;  // <= kThreads
  const int hl = threadIdx.x / lanes, head_lanes = kThreads / lanes;
  const int l = threadIdx.x - hl * lanes;
  const int tk = l / a.units, u = l - tk * a.units;
  if (hl >= head_lanes || tk >= tokens) return;
  const int h0 = blockIdx.y * a.heads_per, h1 = min(h0 + a.heads_per, a.n_heads);
  const int turning = HALF ? a.R / 16 : a.R / 8;
  const uint16_t* x = a.x + (t0 + tk) * a.xt;
  uint16_t* y = a.y + (t0 + tk) * a.yt;
  constexpr int kU = 4;
  if (u >= turning) {  // passes through
    const int d = a.R + 8 * (u - turning);
    for (int h = h0 + hl; h < h1; h += kU * head_lanes) {
      uint4 v[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (h + k * head_lanes < h1) v[k] = *reinterpret_cast<const uint4*>(x + (h + k * head_lanes) * a.xh + d);
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (h + k * head_lanes < h1) *reinterpret_cast<uint4*>(y + (h + k * head_lanes) * a.yh + d) = v[k];
    }
    return;
  }
  constexpr int kPairs = HALF ? 8 : 4;
  float2 c[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) c[i] = cs[tk * (a.R / 2) + u * kPairs + i];
  const int d1 = 8 * u, d2 = 8 * u + a.R / 2;
  for (int h = h0 + hl; h < h1; h += kU * head_lanes) {
    uint4 v1[kU], v2[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int hh = h + k * head_lanes;
      if (hh < h1) {
        v1[k] = *reinterpret_cast<const uint4*>(x + hh * a.xh + d1);
        if constexpr (HALF) v2[k] = *reinterpret_cast<const uint4*>(x + hh * a.xh + d2);
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int hh = h + k * head_lanes;
      if (hh >= h1) break;
      uint32_t* p = reinterpret_cast<uint32_t*>(&v1[k]);
      if constexpr (HALF) {
        uint32_t* r = reinterpret_cast<uint32_t*>(&v2[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = half_bits_to_float(p[i] & 0xFFFFu), a1 = half_bits_to_float(p[i] >> 16);
          const float b0 = half_bits_to_float(r[i] & 0xFFFFu), b1 = half_bits_to_float(r[i] >> 16);
          p[i] = float_to_half_bits(rope_first(a0, b0, c[2 * i])) |
                 (float_to_half_bits(rope_first(a1, b1, c[2 * i + 1])) << 16);
          r[i] = float_to_half_bits(rope_second(a0, b0, c[2 * i])) |
                 (float_to_half_bits(rope_second(a1, b1, c[2 * i + 1])) << 16);
        }
        *reinterpret_cast<uint4*>(y + hh * a.yh + d2) = v2[k];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = half_bits_to_float(p[i] & 0xFFFFu), b0 = half_bits_to_float(p[i] >> 16);
          p[i] = float_to_half_bits(rope_first(a0, b0, c[i])) | (float_to_half_bits(rope_second(a0, b0, c[i])) << 16);
        }
      }
      *reinterpret_cast<uint4*>(y + hh * a.yh + d1) = v1[k];
    }
  }
}

// Any even R: a place is one pair, or one value that passes through. Taken
// where the pairs' chunks are not 16-byte aligned (HALF with R % 16, or
// INTERLEAVED with R % 8).
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ RopeArgs a, int half_layout) {
  extern __shared__ float2 cs[];
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens_per;
  const int tokens = static_cast<int>(min(static_cast<long long>(a.tokens_per), a.n_tokens - t0));
  fill_table(a, cs, t0, tokens);
  const int h0 = blockIdx.y * a.heads_per, heads = min(a.heads_per, a.n_heads - h0), half = a.R / 2;
  for (int w = threadIdx.x; w < tokens * heads * a.units; w += kThreads) {
    const int u = w % a.units, th = w / a.units, h = h0 + th % heads, tk = th / heads;
    const uint16_t* x = a.x + (t0 + tk) * a.xt + h * a.xh;
    uint16_t* y = a.y + (t0 + tk) * a.yt + h * a.yh;
    if (u >= half) {
      y[a.R + u - half] = x[a.R + u - half];
      continue;
    }
    const int i1 = half_layout ? u : 2 * u, i2 = half_layout ? u + half : 2 * u + 1;
    const float x1 = half_bits_to_float(x[i1]), x2 = half_bits_to_float(x[i2]);
    const float2 c = cs[tk * half + u];
    y[i1] = static_cast<uint16_t>(float_to_half_bits(rope_first(x1, x2, c)));
    y[i2] = static_cast<uint16_t>(float_to_half_bits(rope_second(x1, x2, c)));
  }
}

}  // namespace

exq_status launch_rope(const exq_rope_params& rope, const exq_rows& x, long long n_tokens, int n_heads, int D,
                       const int32_t* pos, const exq_rows& y, bool grad, int sms, cudaStream_t stream) {
  RopeArgs a{};
  a.steps = rope.steps;
  a.pos = pos;
  a.x = x.data;
  a.y = y.data;
  a.xt = x.token_stride;
  a.xh = x.head_stride;
  a.yt = y.token_stride;
  a.yh = y.head_stride;
  a.n_tokens = n_tokens;
  a.n_heads = n_heads;
  a.D = D;
  a.R = rope.R;
  a.gain = rope.gain;
  a.grad = grad;
  const bool half = rope.layout == EXQ_ROPE_HALF;
  const bool vec = rope.R % (half ? 16 : 8) == 0;
  const bool in_place = x.data == y.data;
  if (vec)
    a.units = (half ? rope.R / 16 : rope.R / 8) + (in_place ? 0 : (D - rope.R) / 8);
  else
    a.units = rope.R / 2 + (in_place ? 0 : D - rope.R);
  int tokens = std::max(1, kThreads / (rope.R / 2));
  if (vec) tokens = std::min(tokens, kThreads / a.units);
  // at most 4 tokens a block (8 left a second, part-filled wave of blocks: 77
  // for 54 us at 8000 tokens of 64 half-turned heads; fully turned 50 and 50,
  // 55 with two; 8 heads of 64, 16000 tokens: 37 with four, 28 with eight; 16 of
  // 256, 4000: 26 and 28), fewer while there is not a block for each SM twice
  // over
  tokens = std::min(tokens, 4);
  while (tokens > 1 && n_tokens < 2ll * sms * tokens) tokens /= 2;
  a.tokens_per = tokens;
  const long long gx = (n_tokens + a.tokens_per - 1) / a.tokens_per;
  if (gx > 0x7FFFFFFFll) return EXQ_ERR_UNSUPPORTED;
  // few tokens: the heads are split over blocks until two blocks an SM have work
  const int head_lanes = vec ? std::max(1, kThreads / (a.units * a.tokens_per)) : 1;
  const long long want = std::max(1ll, (2ll * sms + gx - 1) / gx);
  const int splits = static_cast<int>(std::min<long long>(want, (n_heads + head_lanes - 1) / head_lanes));
  a.heads_per = (n_heads + splits - 1) / splits;
  const dim3 grid(static_cast<unsigned>(gx), (n_heads + a.heads_per - 1) / a.heads_per);
  const size_t smem = static_cast<size_t>(a.tokens_per) * (rope.R / 2) * sizeof(float2);
  if (!vec)
    rope_any_kernel<<<grid, kThreads, smem, stream>>>(a, half);
  else if (half)
    rope_kernel<true><<<grid, kThreads, smem, stream>>>(a);
  else
    rope_kernel<false><<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

}  // namespace exq
