// The decode product of the 4-bit format and the expert layer: routing, and
// the launches of the streaming kernel (exq_fp4_stream.cuh).
#include <algorithm>
#include <cstring>

#include "exq_fp4_stream.cuh"

namespace exq {
namespace {

using namespace fp4s;

// ---------------------------------------------------------------- routing

struct PrepareArgs {
  const uint16_t* x;       // [T, D]
  // x's parts for the streaming kernel
  uint32_t* codes;         // [T * 8, D / 2] bytes
  uint32_t* scales;        // tiles, or lines for each [token, unit]
  int split_blocks, k_units;
  // routing, where the layer has a router
  const uint16_t* router;  // [E, D]
  float* logits;           // [T, E]
  int32_t* ids;            // [T, top_k]
  float* weights;
  unsigned* counter;
  int T, D, E, top_k, renorm;
};

constexpr int kPrepareThreads = 256;

// Rows of x as eight 4-bit rows each (see exq_fp4_stream.cuh): a thread takes 8
// values, the 2 or 4 of a block find its scale together, and those of a scale
// word write it to the 8 rows. Blocks past the row's end are written as blocks
// of zeros as far as their scale tile goes: the MMAs read them.
template <int FMT, bool TILES>
__device__ __forceinline__ void split_x(const PrepareArgs& a) {
  constexpr int kBlockThreads = fp4_block(FMT) / 8, kWordThreads = 4 * kBlockThreads;
  const int k_tiles = (a.D + fp4_tile_k(FMT) - 1) / fp4_tile_k(FMT);
  const int row_threads = k_tiles * kWordThreads;
  const int total = a.T * row_threads;
  const int stride = a.split_blocks * kPrepareThreads;
  const int padded = (total + 31) / 32 * 32;  // whole warps
  for (int i = (blockIdx.x * kPrepareThreads) + threadIdx.x; i < padded; i += stride) {
    const int t = i / row_threads, c = i - t * row_threads;
    const bool in = i < total && c * 8 < a.D;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (in) x = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(t) * a.D) + c);
    const uint32_t h[4] = {x.x, x.y, x.z, x.w};
    uint32_t m2 = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, h[j] & 0x7FFF7FFFu);
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
    for (int d = 1; d < kBlockThreads; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const bool bad = m >= 0x7C00u;  // an infinity or a NaN: the block is NaN
    const int e = bad ? 0 : part_exponent<FMT>(__half2float(__ushort_as_half(static_cast<unsigned short>(m))), kXTop);
    const uint32_t byte = bad ? (FMT == EXQ_FP4_E4M3 ? 0x7Fu : 0xFFu) : part_scale_byte<FMT>(e, kXTop);
    const float r = pow2(-e);
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      q[2 * j] = bad ? 0.f : v.x * r;
      q[2 * j + 1] = bad ? 0.f : v.y * r;
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const uint32_t word = e2m1x8(q);
      if (in) a.codes[(static_cast<size_t>(t) * kParts + p) * (a.D / 8) + c] = word;
      const uint32_t v[4] = {e2m1x2_f16<0>(word), e2m1x2_f16<1>(word), e2m1x2_f16<2>(word), e2m1x2_f16<3>(word)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
        q[2 * j] = (q[2 * j] - d.x) * 8.f;
        q[2 * j + 1] = (q[2 * j + 1] - d.y) * 8.f;
      }
    }
    uint32_t word = byte << (8 * ((c / kBlockThreads) & 3));
#pragma unroll
    for (int d = kBlockThreads; d < kWordThreads; d <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, d);
    const int p = c % kWordThreads, tile = c / kWordThreads;
    if (i < total && p < kParts) {
      if constexpr (TILES)
        a.scales[(tile * 512 + fp4_tile_byte(t * kParts + p)) / 4] = word;
      else
        a.scales[((static_cast<size_t>(t) * a.k_units * unit_tiles(FMT) + tile) * kLines + p * 16) / 4] = word;
    }
  }
}

// Routing: one CTA an expert: its row against every token, fp32 sums of exact products
// (a thread's share in order of k, then a tree). The last CTA to finish picks
// each token's experts, a warp a token. The router is small (128 experts x
// 4096: 1 MB): what counts is the way from launch to result.
template <int TT>
__device__ __forceinline__ void route(const PrepareArgs& a) {
  __shared__ float sums[kPrepareThreads / 32][16];
  __shared__ int is_last;
  const int e = blockIdx.x - a.split_blocks, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.f;
  const uint16_t* wr = a.router + static_cast<size_t>(e) * a.D;
  for (int k = threadIdx.x * 8; k < a.D; k += kPrepareThreads * 8) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(wr + k));
    const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t >= a.T) break;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(t) * a.D + k));
      const uint32_t xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&wv[j]));
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&xv[j]));
        acc[t] = fmaf(p.x, q.x, acc[t]);
        acc[t] = fmaf(p.y, q.y, acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int d = 16; d; d >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], d);
    if (lane == 0) sums[warp][t] = acc[t];
  }
  __syncthreads();
  if (threadIdx.x < a.T) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kPrepareThreads / 32; ++w) v += sums[w][threadIdx.x];
    __stcg(a.logits + threadIdx.x * a.E + e, v);
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    is_last = atomicAdd(a.counter, 1u) == static_cast<unsigned>(a.E) - 1u;
    if (is_last) *a.counter = 0u;
    __threadfence();
  }
  __syncthreads();
  if (!is_last) return;

  for (int t = warp; t < a.T; t += kPrepareThreads / 32) {
    constexpr int kPer = kMaxExperts / 32;
    float v[kPer];  // lane's logits: experts lane, lane + 32, ...
    unsigned gone = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 32 * i + lane < a.E ? __ldcg(a.logits + t * a.E + 32 * i + lane) : 0.f;
    float top = 0.f, total = 0.f, mine = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
      // the largest left: as unsigned keys that order as the numbers do, a NaN as -infinity
      unsigned key = 0u;
      int at = 1 << 30;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (32 * i + lane >= a.E || (gone >> i & 1u)) continue;
        const unsigned b = v[i] != v[i] ? 0xFF800000u : v[i] == 0.f ? 0u : __float_as_uint(v[i]);
        const unsigned k = b & 0x80000000u ? ~b : b | 0x80000000u;  // above 0 for every number
        if (k > key) { key = k; at = 32 * i + lane; }
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const unsigned k = __shfl_xor_sync(0xffffffffu, key, d);
        const int o = __shfl_xor_sync(0xffffffffu, at, d);
        if (k > key || (k == key && o < at)) { key = k; at = o; }
      }
      float l = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (32 * i + lane == at) { gone |= 1u << i; l = v[i]; }
      l = __shfl_sync(0xffffffffu, l, at & 31);
      if (j == 0) top = l;
      const float p = expf(l - top);
      if (lane == j) mine = p;
      total += p;
      if (lane == 0) a.ids[t * a.top_k + j] = at;
    }
    if (!a.renorm) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (32 * i + lane < a.E) s += expf(v[i] - top);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      total = s;
    }
    if (lane < a.top_k) a.weights[t * a.top_k + lane] = mine / total;
  }
}

// What comes before the streaming kernel: x's parts (the first blocks), and an
// expert layer's routing (the others).
template <int FMT, bool TILES, int TT>
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const __grid_constant__ PrepareArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (static_cast<int>(blockIdx.x) < a.split_blocks)
    split_x<FMT, TILES>(a);
  else if constexpr (TT > 0)
    route<TT>(a);
}

// ---------------------------------------------------------------- launches

int div_up(int a, int b) { return (a + b - 1) / b; }

exq_status launch_prepare(int format, bool tiles, PrepareArgs p, cudaStream_t stream) {
  const int threads = p.T * div_up(p.D, fp4_tile_k(format)) * (fp4_tile_k(format) / 8);
  p.split_blocks = div_up(threads, kPrepareThreads);
  const bool e4m3 = format == EXQ_FP4_E4M3;
  constexpr int A = EXQ_FP4_E4M3, B = EXQ_FP4_E8M0;
  auto fn = tiles ? (e4m3 ? prepare_kernel<A, true, 0> : prepare_kernel<B, true, 0>)
            : !p.router ? (e4m3 ? prepare_kernel<A, false, 0> : prepare_kernel<B, false, 0>)
            : p.T == 1 ? (e4m3 ? prepare_kernel<A, false, 1> : prepare_kernel<B, false, 1>)
            : p.T <= 4 ? (e4m3 ? prepare_kernel<A, false, 4> : prepare_kernel<B, false, 4>)
                       : (e4m3 ? prepare_kernel<A, false, 16> : prepare_kernel<B, false, 16>);
  fn<<<p.split_blocks + (p.router ? p.E : 0), kPrepareThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

// (each a programmatic dependent of the launch before it)
template <int MODE>
exq_status launch_stream(int format, const CUtensorMap& m0, const CUtensorMap& m1, const CUtensorMap& mx, const Args& a,
                         int ctas, int device, cudaStream_t stream) {
  auto fn = format == EXQ_FP4_E4M3 ? stream_kernel<EXQ_FP4_E4M3, MODE> : stream_kernel<EXQ_FP4_E8M0, MODE>;
  static PerDevice attr[2];
  if (!attr[format == EXQ_FP4_E4M3].once(device, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal) == cudaSuccess;
      }))
    return EXQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(fp4s::kThreads);
  cfg.dynamicSmemBytes = kSmemTotal;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, m0, m1, mx, a) == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

bool encode_codes(CUtensorMap* map, const void* codes, uint64_t rows, int K, int box_rows) {
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, K / 2, rows, K / 2, kUnitK / 2, box_rows,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B);
}

void set_shape(Args& a, int format, int rows, int K) {
  a.rows = rows;
  a.K = K;
  a.row_tiles = div_up(rows, kRows);
  a.k_units = div_up(K, kUnitK);
  a.k_tiles = div_up(K, fp4_tile_k(format));
  const int starve = testing_starve_rounds();
  a.wait_limit = starve > 0 ? starve : kFp4WaitLimit;
  a.starve = starve > 0 ? 1 : 0;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t part_bytes(int mode, int sms) { return static_cast<size_t>(sms) * 2 * part_floats(mode) * 4; }

// what lies where in the workspaces, after the counters
struct GemvPlan {
  size_t codes, scales, part, end;
  GemvPlan(int format, int K, int M, int sms) {
    codes = EXQ_FP4_COUNTER_BYTES;
    scales = codes + round256(static_cast<size_t>(M) * kParts * K / 2);
    part = scales + static_cast<size_t>(div_up(K, fp4_tile_k(format))) * 512;
    end = part + part_bytes(kGemv, sms);
  }
};

struct MoePlan {
  size_t logits, x_codes, x_scales, h_codes, h_scales, part, end;
  MoePlan(const exq_moe_layer& l, int T, int sms) {
    const int D = l.gate.K, I = l.gate.rows;
    const size_t lines = token_lines(l.gate.format), pairs = static_cast<size_t>(T) * l.top_k;
    logits = EXQ_FP4_COUNTER_BYTES;
    x_codes = logits + round256(static_cast<size_t>(T) * l.gate.n_experts * 4);
    x_scales = x_codes + round256(static_cast<size_t>(T) * kParts * D / 2);
    h_codes = x_scales + round256(static_cast<size_t>(T) * div_up(D, kUnitK) * lines);
    h_scales = h_codes + round256(pairs * kParts * I / 2);
    part = h_scales + round256(pairs * div_up(I, kUnitK) * lines);
    end = part + std::max(part_bytes(kUp, sms), part_bytes(kDown, sms));
  }
};

// the last counter is the routing's, the others the tiles'
constexpr int kTileCounters = static_cast<int>(EXQ_FP4_COUNTER_BYTES / 4) - 1;

}  // namespace

size_t fp4_gemv_workspace_bytes(const exq_fp4_matrix& w, int M, int sms) { return GemvPlan(w.format, w.K, M, sms).end; }

bool fp4_gemv_fits(int rows) { return div_up(rows, kRows) <= kTileCounters; }

exq_status launch_fp4_gemv(const exq_fp4_matrix& w, const uint16_t* x, int M, uint16_t* y, void* workspace, int sms,
                           int device, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const GemvPlan plan(w.format, w.K, M, sms);
  CUtensorMap mw, mx;
  if (!encode_codes(&mw, w.codes, w.rows, w.K, kRows) ||
      !encode_codes(&mx, ws + plan.codes, static_cast<uint64_t>(M) * kParts, w.K, kParts))
    return EXQ_ERR_CUDA;
  PrepareArgs p{};
  p.x = x;
  p.codes = reinterpret_cast<uint32_t*>(ws + plan.codes);
  p.scales = reinterpret_cast<uint32_t*>(ws + plan.scales);
  p.T = M;
  p.D = w.K;
  const exq_status st = launch_prepare(w.format, true, p, stream);
  if (st != EXQ_OK) return st;
  Args a{};
  set_shape(a, w.format, w.rows, w.K);
  a.sc0 = w.scales;
  a.x_scales = ws + plan.scales;
  a.y = y;
  a.M = M;
  a.factor = w.factor;
  a.counters = static_cast<unsigned*>(workspace);
  a.part = reinterpret_cast<float*>(ws + plan.part);
  const long long units = static_cast<long long>(a.row_tiles) * a.k_units;
  return launch_stream<kGemv>(w.format, mw, mw, mx, a, static_cast<int>(std::min<long long>(units, sms)), device, stream);
}

size_t moe_workspace_bytes(const exq_moe_layer& l, int T, int sms) { return MoePlan(l, T, sms).end; }

bool moe_fits(const exq_moe_layer& l, int T) {
  const long long experts = std::min(l.gate.n_experts, T * l.top_k);
  return experts * div_up(l.gate.rows, kRows) <= kTileCounters && div_up(l.down.rows, kRows) <= kTileCounters;
}

exq_status launch_moe(const exq_moe_layer& l, const uint16_t* x, int T, int32_t* ids, float* weights, uint16_t* y,
                      void* workspace, int sms, int device, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const MoePlan plan(l, T, sms);
  const int E = l.gate.n_experts, D = l.gate.K, I = l.gate.rows, fmt = l.gate.format;
  unsigned* counters = reinterpret_cast<unsigned*>(ws);
  const uint64_t rows = static_cast<uint64_t>(E);
  CUtensorMap mg, mu, md, mx, mh;
  if (!encode_codes(&mg, l.gate.codes, rows * I, D, kRows) || !encode_codes(&mu, l.up.codes, rows * I, D, kRows) ||
      !encode_codes(&md, l.down.codes, rows * D, I, kRows) ||
      !encode_codes(&mx, ws + plan.x_codes, static_cast<uint64_t>(T) * kParts, D, kParts) ||
      !encode_codes(&mh, ws + plan.h_codes, static_cast<uint64_t>(T) * l.top_k * kParts, I, kParts))
    return EXQ_ERR_CUDA;

  PrepareArgs p{};
  p.x = x;
  p.codes = reinterpret_cast<uint32_t*>(ws + plan.x_codes);
  p.scales = reinterpret_cast<uint32_t*>(ws + plan.x_scales);
  p.k_units = div_up(D, kUnitK);
  p.router = l.router;
  p.logits = reinterpret_cast<float*>(ws + plan.logits);
  p.ids = ids;
  p.weights = weights;
  p.counter = counters + kTileCounters;
  p.T = T;
  p.D = D;
  p.E = E;
  p.top_k = l.top_k;
  p.renorm = l.renorm;
  exq_status st = launch_prepare(fmt, false, p, stream);
  if (st != EXQ_OK) return st;

  Args a{};
  set_shape(a, fmt, I, D);
  a.sc0 = l.gate.scales;
  a.sc1 = l.up.scales;
  a.sc_stride = exq_fp4_scale_bytes(fmt, I, D);
  a.x_scales = ws + plan.x_scales;
  a.h_codes = ws + plan.h_codes;
  a.h_scales = ws + plan.h_scales;
  a.h_units = div_up(I, kUnitK);
  a.f0 = l.gate.factors;
  a.f1 = l.up.factors;
  a.ids = ids;
  a.weights = weights;
  a.M = T;
  a.top_k = l.top_k;
  a.n_experts = E;
  a.act = l.act;
  a.counters = counters;
  a.part = reinterpret_cast<float*>(ws + plan.part);
  if ((st = launch_stream<kUp>(fmt, mg, mu, mx, a, sms, device, stream)) != EXQ_OK) return st;

  set_shape(a, fmt, D, I);
  a.sc0 = l.down.scales;
  a.sc1 = nullptr;
  a.sc_stride = exq_fp4_scale_bytes(fmt, D, I);
  a.x_scales = ws + plan.h_scales;
  a.f0 = l.down.factors;
  a.f1 = nullptr;
  a.y = y;
  return launch_stream<kDown>(fmt, md, md, mh, a, sms, device, stream);
}

unsigned take_fp4_stream_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_stream_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_stream_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
