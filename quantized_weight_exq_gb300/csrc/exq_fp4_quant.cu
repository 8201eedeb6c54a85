// fp16 rows to the microscaled 4-bit format and back.
//
// Both ways are bound by memory: 2 bytes a value on the one side, 9/16 (E4M3)
// or 17/32 (E8M0) on the other. A thread takes 16 consecutive values (32 bytes
// in two loads, 8 bytes of codes), so that a warp reads 1 KB in one piece; the
// scale bytes of 4 blocks of a row leave as one 4-byte word of their tile.
#include "exq_fp4.cuh"

namespace exq {
namespace {

constexpr int kThreads = 256;

// magnitude (1..7) -> the tie between it and the code below
__device__ __forceinline__ float tie_below(int c) {
  // 0.25 0.75 1.25 1.75 2.5 3.5 5
  return c <= 4 ? 0.5f * c - 0.25f : c == 5 ? 2.5f : c == 6 ? 3.5f : 5.0f;
}

// The e4m3 byte nearest to a / (6 f), ties to even, at least 1 for a > 0. The
// quotient by a rounded reciprocal is off by less than 2^-21 of itself: where
// the two ends of that range give one byte it is the right one, else the two
// are neighbours and the sign of a - 6 f mid, exact in one fma (6 mid has at
// most 7 bits), decides.
__device__ __forceinline__ uint32_t scale_byte(float a, float f, float inv6f) {
  if (a == 0.f) return 0u;
  const float u = a * inv6f;
  const uint32_t both = e4m3x2(u * (1.f + 0x1p-20f), u * (1.f - 0x1p-20f));
  uint32_t lo = both & 0xFFu, hi = both >> 8;
  if (lo != hi) {
    const float mid = 0.5f * (e4m3_f32(lo) + e4m3_f32(hi));
    const float d = __fmaf_rn(-6.f * mid, f, a);
    lo = d > 0.f ? hi : d < 0.f ? lo : (lo & 1u) ? hi : lo;
  }
  return max(lo, 1u);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const uint4* __restrict__ x, uint2* __restrict__ codes,
                                                            uint32_t* __restrict__ scales, int rows, int K, float f,
                                                            float inv6f) {
  constexpr int kPer = fp4_tile_k(FMT) / 16;  // threads of one scale word: 4 or 8
  const int words = (K + fp4_tile_k(FMT) - 1) / fp4_tile_k(FMT);
  const long long padded = static_cast<long long>((rows + 127) / 128) * 128;
  const long long total = padded * words * kPer;
  const int pieces = K / 16;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    // total is a multiple of 32 (padded is one of 128): the warp is whole here
    const long long row = i / (words * kPer);
    const int piece = static_cast<int>(i - row * (words * kPer));
    const bool in = row < rows && piece < pieces;
    uint32_t h[8] = {};
    if (in) {
      const uint4* src = x + (row * pieces + piece) * 2;
      const uint4 p = __ldcs(src), q = __ldcs(src + 1);
      h[0] = p.x; h[1] = p.y; h[2] = p.z; h[3] = p.w;
      h[4] = q.x; h[5] = q.y; h[6] = q.z; h[7] = q.w;
    }
    // the largest magnitude, as bits: they order as the numbers do, infinity and NaN above
    uint32_t m2 = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, h[j] & 0x7FFF7FFFu);
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if constexpr (FMT == EXQ_FP4_E8M0) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const bool finite = m < 0x7C00u;
    const float a = finite ? __half2float(__ushort_as_half(static_cast<unsigned short>(m))) : 0.f;

    uint32_t byte, c0, c1;
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      v[2 * j] = t.x;
      v[2 * j + 1] = t.y;
    }
    if constexpr (FMT == EXQ_FP4_E4M3) {
      byte = finite ? scale_byte(a, f, inv6f) : 0x7Fu;
      const float s = e4m3_f32(byte);
      const float r = a > 0.f ? 1.f / (s * f) : 0.f;
      // as for the scale: a code that both ends of the quotient's range give is right
      const float rl = r * (1.f - 0x1p-20f), rh = r * (1.f + 0x1p-20f);
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) { lo[j] = v[j] * rl; hi[j] = v[j] * rh; }
      c0 = e2m1x8(lo);
      uint32_t d0 = c0 ^ e2m1x8(hi);
#pragma unroll
      for (int j = 0; j < 8; ++j) { lo[j] = v[8 + j] * rl; hi[j] = v[8 + j] * rh; }
      c1 = e2m1x8(lo);
      uint32_t d1 = c1 ^ e2m1x8(hi);
      if (d0 | d1) {
        // the code is the lower one's or the next: the sign of |x| - tie s f, exact in one fma
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int sh = 4 * (j & 7);
          const uint32_t d = ((j < 8 ? d0 : d1) >> sh) & 0xFu;
          if (d) {
            const uint32_t c = ((j < 8 ? c0 : c1) >> sh) & 7u;
            const float e = __fmaf_rn(-tie_below(static_cast<int>(c) + 1) * s, f, fabsf(v[j]));
            if (e > 0.f || (e == 0.f && (c & 1u))) (j < 8 ? c0 : c1) += 1u << sh;
          }
        }
      }
    } else {
      // floor(log2 a) from the bits: fp16 subnormals by their leading one
      const int top = m >= 0x400u ? static_cast<int>(m >> 10) - 15 : 31 - __clz(static_cast<int>(m)) - 24;
      const int e = m == 0u ? -127 : top - 2;  // at least -26 otherwise
      byte = finite ? static_cast<uint32_t>(e + 127) : 0xFFu;
      const float r = __uint_as_float(static_cast<uint32_t>(127 - max(e, -126)) << 23);  // a power of two: exact
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = v[j] * r;
      c0 = e2m1x8(q);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = v[8 + j] * r;
      c1 = e2m1x8(q);
    }
    if (!finite) c0 = c1 = 0u;
    if (in) codes[row * pieces + piece] = make_uint2(c0, c1);

    // the word's four bytes to its first thread
    if (!in) byte = 0u;
    uint32_t word;
    if constexpr (FMT == EXQ_FP4_E4M3) {
      word = byte | (__shfl_down_sync(0xffffffffu, byte, 1) << 8);
      word |= __shfl_down_sync(0xffffffffu, word, 2) << 16;
    } else {
      word = byte | (__shfl_down_sync(0xffffffffu, byte, 2) << 8);
      word |= __shfl_down_sync(0xffffffffu, word, 4) << 16;
    }
    if (piece % kPer == 0) {
      const int r = static_cast<int>(row & 127);
      const long long tile = (row >> 7) * words + piece / kPer;
      scales[(tile * 512 + fp4_tile_byte(r)) / 4] = word;
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint2* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              uint4* __restrict__ out, int rows, int K, float f) {
  const int words = (K + fp4_tile_k(FMT) - 1) / fp4_tile_k(FMT);
  const int pieces = K / 16;
  const long long total = static_cast<long long>(rows) * pieces;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long row = i / pieces;
    const int piece = static_cast<int>(i - row * pieces);
    const int block = FMT == EXQ_FP4_E4M3 ? piece : piece >> 1;
    const uint2 c = __ldcs(codes + i);
    const uint32_t b = __ldg(scales + ((row >> 7) * words + (block >> 2)) * 512 + fp4_tile_byte(static_cast<int>(row & 127)) +
                             (block & 3));
    const float s = FMT == EXQ_FP4_E4M3 ? e4m3_f32(b) : e8m0_f32(b);
    const uint32_t p[8] = {e2m1x2_f16<0>(c.x), e2m1x2_f16<1>(c.x), e2m1x2_f16<2>(c.x), e2m1x2_f16<3>(c.x),
                           e2m1x2_f16<0>(c.y), e2m1x2_f16<1>(c.y), e2m1x2_f16<2>(c.y), e2m1x2_f16<3>(c.y)};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p[j]));
      // code times scale is exact (6 bits), the factor rounds once in fp32
      const __half2 y = __floats2half2_rn(v.x * s * f, v.y * s * f);
      o[j] = *reinterpret_cast<const uint32_t*>(&y);
    }
    __stcs(out + 2 * i, make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(out + 2 * i + 1, make_uint4(o[4], o[5], o[6], o[7]));
  }
}

int blocks_for(long long threads, int sms) {
  const long long b = (threads + kThreads - 1) / kThreads;
  return static_cast<int>(b < 16LL * sms ? b : 16LL * sms);
}

}  // namespace

exq_status launch_fp4_quantize(const uint16_t* x, const exq_fp4_matrix& m, int sms, cudaStream_t stream) {
  const int words = (m.K + fp4_tile_k(m.format) - 1) / fp4_tile_k(m.format);
  const long long threads = static_cast<long long>((m.rows + 127) / 128) * 128 * words * (fp4_tile_k(m.format) / 16);
  auto fn = m.format == EXQ_FP4_E4M3 ? quantize_kernel<EXQ_FP4_E4M3> : quantize_kernel<EXQ_FP4_E8M0>;
  fn<<<blocks_for(threads, sms), kThreads, 0, stream>>>(
      reinterpret_cast<const uint4*>(x), reinterpret_cast<uint2*>(m.codes), reinterpret_cast<uint32_t*>(m.scales), m.rows, m.K,
      m.factor, 1.f / (6.f * m.factor));
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

exq_status launch_fp4_dequantize(const exq_fp4_matrix& m, uint16_t* out, int sms, cudaStream_t stream) {
  auto fn = m.format == EXQ_FP4_E4M3 ? dequantize_kernel<EXQ_FP4_E4M3> : dequantize_kernel<EXQ_FP4_E8M0>;
  fn<<<blocks_for(static_cast<long long>(m.rows) * (m.K / 16), sms), kThreads, 0, stream>>>(
      reinterpret_cast<const uint2*>(m.codes), m.scales, reinterpret_cast<uint4*>(out), m.rows, m.K, m.factor);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

}  // namespace exq
