// fp16 rows to the microscaled 4-bit format and back.
//
// Both ways are bound by memory: 2 bytes a value on the one side, 9/16 (E4M3)
// or 17/32 (E8M0) on the other. A quantising thread takes 16 consecutive
// values (one load of 32 bytes, 8 bytes of codes), so that a warp reads 1 KB in
// one piece; the scale bytes of 4 blocks of a row leave as one 4-byte word of
// their tile. 28672 x 8192, E8M0: 90 us there and 94 back, 6.4 TB/s; E4M3: 111
// there, 130 where many values are ties (a factor of 0.025).
#include "exq_fp4.cuh"

namespace exq {
namespace {

constexpr int kThreads = 256;

// Both kernels are launched while the one before them may still run, and let
// the next do so; nothing is read or written before it is over.
__device__ __forceinline__ void begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// magnitude (1..7) -> the tie between it and the code below
__device__ __forceinline__ float tie_below(int c) {
  // 0.25 0.75 1.25 1.75 2.5 3.5 5
  return c <= 4 ? 0.5f * c - 0.25f : c == 5 ? 2.5f : c == 6 ? 3.5f : 5.0f;
}

// A number of 64 bits as the sum of three of 32: 24, 24 and 5 bits.
struct Divisor {
  float h, m, l;
};

// What an E4M3 matrix's factor f is to the quantiser. s f is rounded to 64
// bits: a scale s is one of 8 numbers in [1, 2) times a power of two, with which
// the product scales exactly.
struct Factor {
  float f, inv6f;
  Divisor six;       // 6 f
  Divisor times[8];  // (1 + i / 8) f
};

// Whether v / d, rounded to 64 bits, goes to the number above the tie t and not
// to the one below, which is `odd` or even; t has at most 5 bits, v / d is within
// 2^-18 of it. The quotient rounds to t where it is within half a step of t,
// whose last bit is even: v - t d is compared with half a step times d. (Below a
// power of two a step is half as long, but no tie above an odd number is one.)
// In fp32, whose units are many: e has the sign of v - t d, and is v - t d where
// that is below 2^-33 of v. The first difference has 11 bits (t h has 29, and 18
// cancel), the second is rounded only where the third cannot change its sign,
// the third only where it is far above the last bits of d. (Of an f of 32 bits a
// difference is zero or above 2^-34 of v: the exact quotient decides.)
__device__ __forceinline__ bool rounds_up(float v, float t, const Divisor& d, bool odd) {
  const float e = __fmaf_rn(-t, d.l, __fmaf_rn(-t, d.m, __fmaf_rn(-t, d.h, v)));
  const float half = __uint_as_float((__float_as_uint(t) & 0x7F800000u) - (53u << 23));
  const float w = odd ? half : -half;
  const float over = __fmaf_rn(w, d.m, __fmaf_rn(w, d.h, e));
  return odd ? over >= 0.f : over > 0.f;
}

// The e4m3 byte nearest to a / (6 f), ties to even, at least 1 for a > 0. The
// quotient in 32 bits by a rounded reciprocal is off by less than 2^-21 of
// itself: where the two ends of that range give one byte it is the right one,
// else the two are neighbours and what lies between them decides.
__device__ __forceinline__ uint32_t scale_byte(float a, const Factor& f) {
  if (a == 0.f) return 0u;
  const float u = a * f.inv6f;
  const uint32_t both = e4m3x2(u * (1.f + 0x1p-20f), u * (1.f - 0x1p-20f));
  uint32_t lo = both & 0xFFu, hi = both >> 8;
  if (lo != hi) {
    const float mid = 0.5f * (e4m3_f32(lo) + e4m3_f32(hi));
    if (rounds_up(a, mid, f.six, lo & 1u)) lo = hi;
  }
  return max(lo, 1u);
}

// Row and piece of an index that goes up by a fixed stride: a division at the
// start only (of 64-bit numbers, 100 instructions).
struct Walk {
  long long row, d_row;
  int piece, d_piece, per_row;
  __device__ __forceinline__ Walk(long long i, long long stride, int n) : per_row(n) {
    row = i / n;
    piece = static_cast<int>(i - row * n);
    d_row = stride / n;
    d_piece = static_cast<int>(stride - d_row * n);
  }
  __device__ __forceinline__ void next() {
    row += d_row;
    piece += d_piece;
    if (piece >= per_row) {
      piece -= per_row;
      ++row;
    }
  }
};

// (Six blocks an SM, 40 registers: with 44 E4M3 takes 122 us, not 111.)
template <int FMT>
__global__ void __launch_bounds__(kThreads, 6) quantize_kernel(const uint16_t* __restrict__ x, uint2* __restrict__ codes,
                                                               uint32_t* __restrict__ scales, int rows, int K, bool wide,
                                                               const __grid_constant__ Factor f) {
  constexpr int kPer = fp4_tile_k(FMT) / 16;  // threads of one scale word: 4 or 8
  begin();
  const int words = (K + fp4_tile_k(FMT) - 1) / fp4_tile_k(FMT);
  const long long padded = static_cast<long long>((rows + 127) / 128) * 128;
  const int per_row = words * kPer;
  const long long total = padded * per_row;
  const int pieces = K / 16;
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  Walk at(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, stride, per_row);
  // total is a multiple of 32 (padded is one of 128): the warp is whole here
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += stride, at.next()) {
    const long long row = at.row;
    const int piece = at.piece;
    const bool in = row < rows && piece < pieces;
    uint32_t h[8] = {};
    if (in) {
      const uint16_t* src = x + (row * pieces + piece) * 16;
      if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]), "=r"(h[4]), "=r"(h[5]), "=r"(h[6]), "=r"(h[7])
                     : "l"(src));
      } else {
        const uint4 p = __ldcs(reinterpret_cast<const uint4*>(src)), q = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
        h[0] = p.x; h[1] = p.y; h[2] = p.z; h[3] = p.w;
        h[4] = q.x; h[5] = q.y; h[6] = q.z; h[7] = q.w;
      }
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
      byte = finite ? scale_byte(a, f) : 0x7Fu;
      const float s = e4m3_f32(byte);
      const float r = a > 0.f ? 1.f / (s * f.f) : 0.f;
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
        // the code is the lower one's or the next
        const uint32_t bits = __float_as_uint(s);
        const Divisor& d = f.times[(bits >> 20) & 7u];
        const float power = __uint_as_float(bits & 0x7F800000u);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int sh = 4 * (j & 7);
          if (((j < 8 ? d0 : d1) >> sh) & 0xFu) {
            const uint32_t c = ((j < 8 ? c0 : c1) >> sh) & 7u;
            if (rounds_up(fabsf(v[j]), tie_below(static_cast<int>(c) + 1) * power, d, c & 1u)) (j < 8 ? c0 : c1) += 1u << sh;
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

// 32 codes of a row, their scales and where they go
template <int FMT>
struct Codes32 {
  uint4 c;
  uint32_t s;  // E4M3: the bytes of two blocks; E8M0: of one
  uint16_t* to;
  __device__ __forceinline__ void load(const uint4* codes, const uint8_t* scales, uint16_t* out, long long i, const Walk& at,
                                       int words) {
    c = __ldcs(codes + i);
    const uint8_t* tile = scales + fp4_tile_byte(static_cast<int>(at.row & 127));
    if constexpr (FMT == EXQ_FP4_E4M3)
      s = __ldg(reinterpret_cast<const uint16_t*>(tile + ((at.row >> 7) * words + (at.piece >> 1)) * 512 + (at.piece & 1) * 2));
    else
      s = __ldg(tile + ((at.row >> 7) * words + (at.piece >> 2)) * 512 + (at.piece & 3));
    to = out + 32 * i;
  }
  __device__ __forceinline__ void store(float f, bool wide) const {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float sc = FMT == EXQ_FP4_E4M3 ? e4m3_f32((s >> (8 * h)) & 0xFFu) : e8m0_f32(s);
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t v = w[2 * h + j];
        const uint32_t p[4] = {e2m1x2_f16<0>(v), e2m1x2_f16<1>(v), e2m1x2_f16<2>(v), e2m1x2_f16<3>(v)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&p[k]));
          // code times scale is exact (6 bits), the factor rounds once in fp32
          const __half2 y = __floats2half2_rn(x.x * sc * f, x.y * sc * f);
          o[4 * j + k] = *reinterpret_cast<const uint32_t*>(&y);
        }
      }
      if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 16 * h), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
      } else {
        __stcs(reinterpret_cast<uint4*>(to + 16 * h), make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4*>(to + 16 * h) + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
};

// A thread takes 32 codes at a time (16 bytes; 64 of results, in stores of 32
// bytes, whole sectors), and has the next 32 on their way.
template <int FMT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint4* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              uint16_t* __restrict__ out, int rows, int K, float f, bool wide) {
  begin();
  const int words = (K + fp4_tile_k(FMT) - 1) / fp4_tile_k(FMT);
  const int pieces = K / 32;
  const long long total = static_cast<long long>(rows) * pieces, stride = static_cast<long long>(gridDim.x) * kThreads;
  long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  Walk at(i, stride, pieces);
  for (; i < total; i += 2 * stride) {
    Codes32<FMT> a, b;
    a.load(codes, scales, out, i, at, words);
    at.next();
    const bool two = i + stride < total;
    if (two) b.load(codes, scales, out, i + stride, at, words);
    at.next();
    a.store(f, wide);
    if (two) b.store(f, wide);
  }
}

// whether rows of 32-byte pieces from here can be read and written by the piece (16 bytes are what is asked of callers)
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

Divisor split(double d) {
  Divisor r;
  r.h = static_cast<float>(d);
  r.m = static_cast<float>(d - r.h);
  r.l = static_cast<float>(d - r.h - r.m);
  return r;
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
  Factor f;
  f.f = static_cast<float>(m.factor);
  f.inv6f = static_cast<float>(1. / (6. * m.factor));
  f.six = split(6. * m.factor);
  for (int i = 0; i < 8; ++i) f.times[i] = split((1. + i / 8.) * m.factor);
  return launch_dependent(fn, blocks_for(threads, sms), kThreads, 0, stream, x, reinterpret_cast<uint2*>(m.codes),
                          reinterpret_cast<uint32_t*>(m.scales), m.rows, m.K, aligned32(x), f);
}

exq_status launch_fp4_dequantize(const exq_fp4_matrix& m, uint16_t* out, int sms, cudaStream_t stream) {
  auto fn = m.format == EXQ_FP4_E4M3 ? dequantize_kernel<EXQ_FP4_E4M3> : dequantize_kernel<EXQ_FP4_E8M0>;
  return launch_dependent(fn, blocks_for(static_cast<long long>(m.rows) * (m.K / 32), sms), kThreads, 0, stream,
                          reinterpret_cast<const uint4*>(m.codes), static_cast<const uint8_t*>(m.scales), out, m.rows, m.K,
                          static_cast<float>(m.factor), aligned32(out));
}

}  // namespace exq
