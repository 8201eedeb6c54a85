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
  uint32_t* scales;        // gemv: the parts' scale tiles
  uint8_t* pieces;         // experts: [rows, units]
  const float* h;          // instead of x: [T, D] in fp32,
  unsigned* h_most;        // and each row's largest magnitude (zeroed by the launch that splits x)
  int split_blocks, k_units, pairs;
  // routing, where the layer has a router
  const uint16_t* router;  // [E, D]
  float* logits;           // [T, E]
  int32_t* ids;            // [T, top_k]
  float* weights;
  unsigned* counter;
  int T, D, E, top_k, renorm;
};

constexpr int kPrepareThreads = 512;
constexpr int kSplitThreads = 128;   // of h: their registers fit beside a CTA of the streaming kernel, which need not wait for them

// Rows as eight 4-bit rows each (see exq_fp4_stream.cuh): a thread takes 8
// values, the 2 or 4 of a block find its scale together, and those of a scale
// word write it to the 8 rows. What lies past the row's end is written as
// zeros as far as its scale tile (the MMAs read it) or its unit (no copy
// fills it up) goes. H: rows of h, divided by the power of two of each.
template <int FMT, bool TILES, bool H>
__device__ __forceinline__ void split_rows(const PrepareArgs& a) {
  constexpr int kThreads = H ? kSplitThreads : kPrepareThreads;
  constexpr int kWordThreads = fp4_tile_k(FMT) / 8;
  constexpr int kTop = H ? kHTop : kXTop;
  const int row_threads = TILES ? (a.D + fp4_tile_k(FMT) - 1) / fp4_tile_k(FMT) * kWordThreads : a.k_units * (kUnitK / 8);
  const int total = a.T * row_threads;            // below 2^31: K is, by the entry points, at most 2^25
  const int padded = (total + 31) / 32 * 32;      // whole warps
  for (int i = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x; i < padded; i += a.split_blocks * kThreads) {
    const int t = i / row_threads, c = i - t * row_threads;
    const bool in = i < total && c * 8 < a.D;
    float q[8] = {};
    if (in) {
      if constexpr (H) {
        const float4* src = reinterpret_cast<const float4*>(a.h + static_cast<size_t>(t) * a.D + 8 * c);
        const float4 u = __ldcg(src), v = __ldcg(src + 1);
        const float r = h_scale(__ldcg(a.h_most + t));
        q[0] = u.x * r; q[1] = u.y * r; q[2] = u.z * r; q[3] = u.w * r;
        q[4] = v.x * r; q[5] = v.y * r; q[6] = v.z * r; q[7] = v.w * r;
      } else {
        to_f32(__ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(t) * a.D) + c), q);
      }
    }
    uint32_t words[kParts], word;
    split8<FMT>(q, kTop, c, words, word);
    uint8_t* piece = nullptr;
    if constexpr (!TILES) piece = a.pieces + (static_cast<size_t>(t) * a.k_units + c / (kUnitK / 8)) * piece_bytes(FMT);
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if constexpr (TILES) {
        if (in) a.codes[(static_cast<size_t>(t) * kParts + p) * (a.D / 8) + c] = words[p];
      } else {
        if (i < total) *reinterpret_cast<uint32_t*>(piece + piece_word(p, 8 * c % kUnitK)) = words[p];
      }
    }
    const int p = c % kWordThreads, tile = c / kWordThreads;
    if (i < total && p < kParts) {
      if constexpr (TILES)
        a.scales[(static_cast<size_t>(tile) * 512 + fp4_tile_byte(t * kParts + p)) / 4] = word;
      else
        *reinterpret_cast<uint32_t*>(piece + 1024 + tile % unit_tiles(FMT) * kLines + p * 16) = word;
    }
  }
}

// a logit as an unsigned key that orders as the numbers do, a NaN as -infinity, -0 as 0
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = v != v ? 0xFF800000u : v == 0.f ? 0u : __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Routing: one CTA an expert: its row against every token, fp32 sums of exact products
// (a thread's share in order of k, then a tree). The last CTA to finish picks
// each token's experts. The router is small (128 experts x
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
    uint4 x[TT];  // all on their way at once (rows past the last are the last)
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(min(t, a.T - 1)) * a.D + k));
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint32_t xv[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&wv[j]));
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&xv[j]));
        acc[t] = fmaf(p.x, q.x, acc[t]);
        acc[t] = fmaf(p.y, q.y, acc[t]);
      }
    }
  }
  // the warp's sums: the lanes halve what tokens they have from step to step (one token at a time takes five shuffles each)
  int d = 16;
#pragma unroll
  for (int n = TT / 2; n; n >>= 1, d >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int t = 0; t < n; ++t) {
      const float give = upper ? acc[t] : acc[t + n], keep = upper ? acc[t + n] : acc[t];
      acc[t] = keep + __shfl_xor_sync(0xffffffffu, give, d);
    }
  }
#pragma unroll
  for (; d; d >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], d);
  if (lane % (32 / TT) == 0) sums[warp][lane / (32 / TT)] = acc[0];
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

  // Each expert's place is the number of those before it: larger ones, and equal ones of a lower index. All experts of some
  // tokens are compared with all at once, which for up to 128 of them is sooner done than top_k searches one after the other
  // (3 us, with the loads of code that runs once). Beyond that these comparisons, T E^2 in one CTA, are most of a small layer: 16
  // tokens' routing adds 6, 16, 50 and 177 us with 64, 128, 256 and 512 experts, one token's 2, 3, 5 and 13 (D = 2048).
  constexpr int kHeld = 1024;
  __shared__ unsigned held[kHeld];    // keys of a batch of tokens
  __shared__ float chosen[16][16];
  const int batch = max(1, min(a.T, kHeld / a.E));
  for (int t0 = 0; t0 < a.T; t0 += batch) {
    const int n = min(batch, a.T - t0) * a.E;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPrepareThreads) held[i] = order_key(__ldcg(a.logits + t0 * a.E + i));
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPrepareThreads) {
      const int t = i / a.E, e = i - t * a.E;
      const unsigned key = held[i];
      const unsigned* others = held + t * a.E;
      int place = 0;
#pragma unroll 8
      for (int o = 0; o < a.E; ++o) place += others[o] > key || (others[o] == key && o < e) ? 1 : 0;
      if (place < a.top_k) {
        a.ids[(t0 + t) * a.top_k + place] = e;
        chosen[t0 + t][place] = __ldcg(a.logits + (t0 + t) * a.E + e);
      }
    }
  }
  __syncthreads();
  for (int t = warp; t < a.T; t += kPrepareThreads / 32) {
    const float top = chosen[t][0];
    const float p = lane < a.top_k ? expf(chosen[t][lane] - top) : 0.f;
    float total = p;
    if (!a.renorm) {
      total = 0.f;
      for (int e = lane; e < a.E; e += 32) total += expf(__ldcg(a.logits + t * a.E + e) - top);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane < a.top_k) a.weights[t * a.top_k + lane] = p / total;
  }
}

// What comes before the streaming kernel: x's parts (the first blocks), and an
// expert layer's routing (the others).
template <int FMT, bool TILES, int TT>
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const __grid_constant__ PrepareArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (not sooner: the launch after this reads weights, which may come from the one before this, without another wait)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (static_cast<int>(blockIdx.x) < a.split_blocks) {
    if (!TILES && blockIdx.x == 0)
      for (int i = threadIdx.x; i < a.pairs; i += kPrepareThreads) a.h_most[i] = 0u;
    split_rows<FMT, TILES, false>(a);
  } else if constexpr (TT > 0) {
    route<TT>(a);
  }
}

// Between the experts' products: h's parts. (Places that nothing was written
// to are split all the same; nobody reads them.)
template <int FMT>
__global__ void __launch_bounds__(kSplitThreads) split_h_kernel(const __grid_constant__ PrepareArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the launch after this may start: what it reads before it waits is older than the launch before this
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  split_rows<FMT, false, true>(a);
}

// ---------------------------------------------------------------- launches

int div_up(int a, int b) { return (a + b - 1) / b; }

// A small kernel runs on SMs whose shared memory is set up as the streaming
// kernel wants it: else an SM has to fall idle before that one's CTA may start
// (the experts' down product began 10 us after up's end, not 3).
bool beside_streaming(void (*fn)(PrepareArgs)) {
  return cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) == cudaSuccess;
}

// blocks that split rows of D values, a thread 8 of them
int split_blocks_for(int format, bool tiles, int rows, int D, int threads) {
  const int k = tiles ? fp4_tile_k(format) : kUnitK;
  return std::min(div_up(rows * div_up(D, k) * (k / 8), threads), 8192);
}

exq_status launch_prepare(int format, bool tiles, PrepareArgs p, cudaStream_t stream) {
  p.split_blocks = split_blocks_for(format, tiles, p.T, p.D, kPrepareThreads);
  const bool e4m3 = format == EXQ_FP4_E4M3;
  constexpr int A = EXQ_FP4_E4M3, B = EXQ_FP4_E8M0;
  auto fn = tiles ? (e4m3 ? prepare_kernel<A, true, 0> : prepare_kernel<B, true, 0>)
            : !p.router ? (e4m3 ? prepare_kernel<A, false, 0> : prepare_kernel<B, false, 0>)
            : p.T == 1 ? (e4m3 ? prepare_kernel<A, false, 1> : prepare_kernel<B, false, 1>)
            : p.T <= 4 ? (e4m3 ? prepare_kernel<A, false, 4> : prepare_kernel<B, false, 4>)
            : p.T <= 8 ? (e4m3 ? prepare_kernel<A, false, 8> : prepare_kernel<B, false, 8>)
                       : (e4m3 ? prepare_kernel<A, false, 16> : prepare_kernel<B, false, 16>);
  if (!beside_streaming(fn)) return EXQ_ERR_CUDA;
  return launch_dependent(fn, p.split_blocks + (p.router ? p.E : 0), kPrepareThreads, 0, stream, p);
}

exq_status launch_split_h(int format, PrepareArgs p, cudaStream_t stream) {
  p.split_blocks = split_blocks_for(format, false, p.T, p.D, kSplitThreads);
  auto fn = format == EXQ_FP4_E4M3 ? split_h_kernel<EXQ_FP4_E4M3> : split_h_kernel<EXQ_FP4_E8M0>;
  if (!beside_streaming(fn)) return EXQ_ERR_CUDA;
  return launch_dependent(fn, p.split_blocks, kSplitThreads, 0, stream, p);
}

// Whether the streaming kernel splits the rows itself: one always, and up to
// eight of x where a CTA has few units. The launch that splits them takes 0.5
// to 3.5 us; splitting a row in every CTA takes each of its units up to 60 ns
// longer. Both sides, us, here and by a launch, at (units, rows times units) of a
// CTA: 4 x 1024 x 8192 (1.7, 7) 7.7 and 11.2, 4 x 4096 x 3584 (2.9, 12) 8.2 and 9.2, 2 x 4096 x 11008 (9.1, 18) 11.2 and
// 11.7, 6 x 4096 x 4096 (3.4, 20.2) 8.7 and 9.3, 4 x 4096 x 6656 (5.5, 22) 10.0 and
// 10.8, 8 x 2048 x 6912 (2.8, 23) 9.4 and 10.2, 3 x 11008 x 3584 (7.9, 23.8) 11.7
// and 11.8; 2 x 8192 x 6144 (10.1, 20.2) 12.0 and 11.9, 2 x 11008 x 5120 (11.3, 23)
// 13.2 and 12.7, 3 x 8192 x 5120 (8.4, 25) 11.6 and 11.4, 4 x 8192 x 4096 (6.7,
// 27) 11.2 and 10.8, 8 x 8192 x 5120 (8.4, 67) 14.9 and 12.0. One token of 8 of
// 128 experts of 1536 x 4096: 36.9 and 39.5 us; two and more tokens of other
// layers gained as often as they lost.
bool splits(int mode, int M, long long units, int ctas) {
  return M == 1 || (mode == kGemv && M <= 8 && units <= 10ll * ctas && M * units <= 24ll * ctas);
}

template <int FMT, int MODE, int NT, bool HERE>
exq_status launch_stream(const CUtensorMap& m0, const CUtensorMap& m1, const CUtensorMap& mx, const Args& a, int ctas,
                         int device, cudaStream_t stream) {
  auto fn = stream_kernel<FMT, MODE, NT, HERE>;
  static PerDevice attr;
  if (!attr.once(device, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal) == cudaSuccess;
      }))
    return EXQ_ERR_CUDA;
  return launch_dependent(fn, ctas, threads_of(NT, HERE), kSmemTotal, stream, m0, m1, mx, a);
}

template <int FMT, int MODE>
exq_status launch_stream(bool here, const CUtensorMap& m0, const CUtensorMap& m1, const CUtensorMap& mx, const Args& a, int ctas,
                         int device, cudaStream_t stream) {
  auto go = a.M == 1 ? launch_stream<FMT, MODE, 1, MODE != kUp> : a.M <= 8 ? launch_stream<FMT, MODE, 8, false>
                                                                           : launch_stream<FMT, MODE, 16, false>;
  if constexpr (MODE == kGemv)
    if (here && a.M > 1) go = launch_stream<FMT, MODE, 8, true>;
  return go(m0, m1, mx, a, ctas, device, stream);
}

template <int MODE>
exq_status launch_stream(int format, bool here, const CUtensorMap& m0, const CUtensorMap& m1, const CUtensorMap& mx,
                         const Args& a, int ctas, int device, cudaStream_t stream) {
  return format == EXQ_FP4_E4M3 ? launch_stream<EXQ_FP4_E4M3, MODE>(here, m0, m1, mx, a, ctas, device, stream)
                                : launch_stream<EXQ_FP4_E8M0, MODE>(here, m0, m1, mx, a, ctas, device, stream);
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

// the last counter is the routing's, the others the tiles'
constexpr int kTileCounters = static_cast<int>(EXQ_FP4_COUNTER_BYTES / 4) - 1;

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
  size_t logits, x, h, h_most, h_pieces, part, end;
  MoePlan(const exq_moe_layer& l, int T, int sms) {
    const int D = l.gate.K, I = l.gate.rows;
    const size_t piece = piece_bytes(l.gate.format), pairs = static_cast<size_t>(T) * l.top_k;
    logits = EXQ_FP4_COUNTER_BYTES;
    x = logits + round256(static_cast<size_t>(T) * l.gate.n_experts * 4);
    h = x + round256(static_cast<size_t>(T) * div_up(D, kUnitK) * piece);
    h_most = h + round256(pairs * I * 4);
    h_pieces = h_most + round256(pairs * 4);
    part = h_pieces + round256(pairs * div_up(I, kUnitK) * piece);
    end = part + std::max(part_bytes(kUp, sms), part_bytes(kDown, sms));
  }
};

}  // namespace

size_t fp4_gemv_workspace_bytes(const exq_fp4_matrix& w, int M, int sms) { return GemvPlan(w.format, w.K, M, sms).end; }

bool fp4_gemv_fits(int rows) { return div_up(rows, kRows) <= kTileCounters; }

exq_status launch_fp4_gemv(const exq_fp4_matrix& w, const uint16_t* x, int M, uint16_t* y, void* workspace, int sms,
                           int device, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const GemvPlan plan(w.format, w.K, M, sms);
  CUtensorMap mw, mx;
  if (!encode_codes(&mw, w.codes, w.rows, w.K, kRows)) return EXQ_ERR_CUDA;
  const long long units = static_cast<long long>(div_up(w.rows, kRows)) * div_up(w.K, kUnitK);
  const int ctas = static_cast<int>(std::min<long long>(units, sms));
  const bool here = splits(kGemv, M, units, ctas);
  if (here)
    mx = mw;  // not used
  else if (!encode_codes(&mx, ws + plan.codes, static_cast<uint64_t>(M) * kParts, w.K, M * kParts))
    return EXQ_ERR_CUDA;
  if (!here) {
    PrepareArgs p{};
    p.x = x;
    p.codes = reinterpret_cast<uint32_t*>(ws + plan.codes);
    p.scales = reinterpret_cast<uint32_t*>(ws + plan.scales);
    p.T = M;
    p.D = w.K;
    const exq_status st = launch_prepare(w.format, true, p, stream);
    if (st != EXQ_OK) return st;
  }
  Args a{};
  set_shape(a, w.format, w.rows, w.K);
  a.sc0 = w.scales;
  a.x = ws + plan.scales;
  a.rows_of_x = x;
  a.y = y;
  a.M = M;
  a.factor = static_cast<float>(w.factor);
  a.counters = static_cast<unsigned*>(workspace);
  a.part = reinterpret_cast<float*>(ws + plan.part);
  return launch_stream<kGemv>(w.format, here, mw, mw, mx, a, ctas, device, stream);
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
  CUtensorMap mg, mu, md;
  if (!encode_codes(&mg, l.gate.codes, rows * I, D, kRows) || !encode_codes(&mu, l.up.codes, rows * I, D, kRows) ||
      !encode_codes(&md, l.down.codes, rows * D, I, kRows))
    return EXQ_ERR_CUDA;

  PrepareArgs p{};
  p.x = x;
  p.pieces = ws + plan.x;
  p.h = reinterpret_cast<float*>(ws + plan.h);
  p.h_most = reinterpret_cast<unsigned*>(ws + plan.h_most);
  p.k_units = div_up(D, kUnitK);
  p.pairs = T * l.top_k;
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
  a.x = ws + plan.x;
  a.h = reinterpret_cast<float*>(ws + plan.h);
  a.h_most = reinterpret_cast<unsigned*>(ws + plan.h_most);
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
  a.down_scales = l.down.scales;
  a.down_stride = exq_fp4_scale_bytes(fmt, D, I);
  a.down_row_tiles = div_up(D, kRows);
  a.down_k_units = div_up(I, kUnitK);
  a.down_k_tiles = div_up(I, fp4_tile_k(fmt));
  if ((st = launch_stream<kUp>(fmt, false, mg, mu, md, a, sms, device, stream)) != EXQ_OK) return st;

  const bool here = splits(kDown, T, 0, sms);
  if (!here) {
    p.pieces = ws + plan.h_pieces;
    p.T = T * l.top_k;
    p.D = I;
    p.k_units = div_up(I, kUnitK);
    if ((st = launch_split_h(fmt, p, stream)) != EXQ_OK) return st;
  }

  set_shape(a, fmt, D, I);
  a.sc0 = l.down.scales;
  a.sc1 = nullptr;
  a.sc_stride = exq_fp4_scale_bytes(fmt, D, I);
  a.x = ws + plan.h_pieces;
  a.f0 = l.down.factors;
  a.f1 = nullptr;
  a.y = y;
  return launch_stream<kDown>(fmt, here, md, md, md, a, sms, device, stream);
}

extern "C" int64_t exq_testing_first_unit(int32_t cta, int64_t n_units, int32_t ctas) {
  return ctas >= 1 && cta >= 0 && cta <= ctas && n_units >= ctas ? first_unit(cta, n_units, ctas) : -1;
}

extern "C" int32_t exq_testing_unit_owner(int64_t unit, int64_t n_units, int32_t ctas) {
  return ctas >= 1 && unit >= 0 && unit < n_units && n_units >= ctas ? owner(unit, n_units, ctas) : -1;
}

unsigned take_fp4_stream_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_stream_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_stream_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
