// The decode product of the 4-bit format and the expert layer: routing, and
// the launches of the streaming kernel (exq_fp4_stream.cuh).
#include <algorithm>
#include <cstring>

#include "exq_fp4_stream.cuh"

namespace exq {
namespace {

using namespace fp4s;

// ---------------------------------------------------------------- routing

struct RouteArgs {
  const uint16_t* x;       // [T, D]
  const uint16_t* router;  // [E, D]
  float* logits;           // [T, E]
  int32_t* ids;            // [T, top_k]
  float* weights;
  unsigned* counter;
  int T, D, E, top_k, renorm;
};

constexpr int kRouteThreads = 256;

// One CTA an expert: its row against every token, fp32 sums of exact products
// (a thread's share in order of k, then a tree). The last CTA to finish picks
// each token's experts, a warp a token. The router is small (128 experts x
// 4096: 1 MB): what counts is the way from launch to result.
template <int TT>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ float sums[kRouteThreads / 32][16];
  __shared__ int is_last;
  const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.f;
  const uint16_t* wr = a.router + static_cast<size_t>(e) * a.D;
  for (int k = threadIdx.x * 8; k < a.D; k += kRouteThreads * 8) {
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
    for (int w = 0; w < kRouteThreads / 32; ++w) v += sums[w][threadIdx.x];
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

  for (int t = warp; t < a.T; t += kRouteThreads / 32) {
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

// ---------------------------------------------------------------- launches

int div_up(int a, int b) { return (a + b - 1) / b; }

template <int FMT, int MODE, int NT>
exq_status launch(const CUtensorMap& m0, const CUtensorMap& m1, const Args& a, int ctas, bool dependent, int device,
                  cudaStream_t stream) {
  auto fn = stream_kernel<FMT, MODE, NT>;
  static PerDevice attr;
  if (!attr.once(device, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(MODE, NT)) == cudaSuccess;
      }))
    return EXQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(fp4s::kThreads);
  cfg.dynamicSmemBytes = smem_bytes(MODE, NT);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, m0, m1, a) == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

template <int MODE>
exq_status launch_mode(int format, int M, const CUtensorMap& m0, const CUtensorMap& m1, const Args& a, int ctas,
                       bool dependent, int device, cudaStream_t stream) {
  if (format == EXQ_FP4_E4M3)
    return M <= 8 ? launch<EXQ_FP4_E4M3, MODE, 1>(m0, m1, a, ctas, dependent, device, stream)
                  : launch<EXQ_FP4_E4M3, MODE, 2>(m0, m1, a, ctas, dependent, device, stream);
  return M <= 8 ? launch<EXQ_FP4_E8M0, MODE, 1>(m0, m1, a, ctas, dependent, device, stream)
                : launch<EXQ_FP4_E8M0, MODE, 2>(m0, m1, a, ctas, dependent, device, stream);
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

size_t part_bytes(int mode, int M, int sms) {
  return static_cast<size_t>(sms) * 2 * part_floats(mode, M <= 8 ? 1 : 2) * 4;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// what lies where in exq_moe's workspace, after the counters
struct MoePlan {
  size_t logits, h, part, end;
  MoePlan(const exq_moe_layer& l, int T, int sms) {
    logits = EXQ_FP4_COUNTER_BYTES;
    h = logits + round256(static_cast<size_t>(T) * l.gate.n_experts * 4);
    part = h + round256(static_cast<size_t>(T) * l.top_k * div_up(l.gate.rows, kUnitK) * kHPiece);
    end = part + part_bytes(kUp, T, sms);
  }
};

// the last counter is the routing's, the others the tiles'
constexpr int kTileCounters = static_cast<int>(EXQ_FP4_COUNTER_BYTES / 4) - 1;

}  // namespace

size_t fp4_gemv_workspace_bytes(int M, int sms) { return EXQ_FP4_COUNTER_BYTES + part_bytes(kGemv, M, sms); }

bool fp4_gemv_fits(int rows) { return div_up(rows, kRows) <= kTileCounters; }

exq_status launch_fp4_gemv(const exq_fp4_matrix& w, const uint16_t* x, int M, uint16_t* y, void* workspace, int sms,
                           int device, cudaStream_t stream) {
  CUtensorMap map;
  if (!encode_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K / 2, w.rows, w.K / 2, kUnitK / 2, kRows,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B))
    return EXQ_ERR_CUDA;
  Args a{};
  set_shape(a, w.format, w.rows, w.K);
  a.sc0 = w.scales;
  a.x = x;
  a.out = y;
  a.M = M;
  a.factor = w.factor;
  a.counters = static_cast<unsigned*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + EXQ_FP4_COUNTER_BYTES);
  const long long units = static_cast<long long>(a.row_tiles) * a.k_units;
  return launch_mode<kGemv>(w.format, M, map, map, a, static_cast<int>(std::min<long long>(units, sms)), false, device,
                            stream);
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
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + plan.h);

  CUtensorMap maps[3];
  const exq_fp4_experts* parts[3] = {&l.gate, &l.up, &l.down};
  for (int i = 0; i < 3; ++i)
    if (!encode_2d(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, parts[i]->codes, parts[i]->K / 2,
                   static_cast<uint64_t>(E) * parts[i]->rows, parts[i]->K / 2, kUnitK / 2, kRows,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B))
      return EXQ_ERR_CUDA;

  if (l.router) {
    RouteArgs r{x, l.router, reinterpret_cast<float*>(ws + plan.logits), ids, weights, counters + kTileCounters,
                T, D, E, l.top_k, l.renorm};
    auto fn = T == 1 ? route_kernel<1> : T <= 4 ? route_kernel<4> : route_kernel<16>;
    fn<<<E, kRouteThreads, 0, stream>>>(r);
    if (cudaGetLastError() != cudaSuccess) return EXQ_ERR_CUDA;
  }

  Args a{};
  set_shape(a, fmt, I, D);
  a.sc0 = l.gate.scales;
  a.sc1 = l.up.scales;
  a.sc_stride = exq_fp4_scale_bytes(fmt, I, D);
  a.x = x;
  a.out = h;
  a.h_units = div_up(I, kUnitK);
  a.f0 = l.gate.factors;
  a.f1 = l.up.factors;
  a.f2 = l.down.factors;
  a.ids = ids;
  a.weights = weights;
  a.M = T;
  a.top_k = l.top_k;
  a.n_experts = E;
  a.act = l.act;
  a.counters = counters;
  a.part = reinterpret_cast<float*>(ws + plan.part);
  const exq_status st = launch_mode<kUp>(fmt, T, maps[0], maps[1], a, sms, l.router != nullptr, device, stream);
  if (st != EXQ_OK) return st;

  set_shape(a, fmt, D, I);
  a.sc0 = l.down.scales;
  a.sc1 = nullptr;
  a.sc_stride = exq_fp4_scale_bytes(fmt, D, I);
  a.x = h;
  a.out = y;
  a.factor = 1.f;
  return launch_mode<kDown>(fmt, T, maps[2], maps[2], a, sms, true, device, stream);
}

unsigned take_fp4_stream_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_stream_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_stream_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
