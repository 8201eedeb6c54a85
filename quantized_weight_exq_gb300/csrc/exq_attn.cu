// Attention of new tokens over a paged (quantised) KV cache:
//   o = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q . k_t - m),
// over the cached tokens t a row sees, m the running maximum.
//
// A block does one (row, query head): its warps take cached tokens in turn, a
// lane holding D / 32 values of each, and merge their (m, sum, o) at the end.
#include <cmath>

#include "exq_device.cuh"
#include "exq_internal.h"
#include "exq_rope.cuh"

namespace exq {
namespace {

__device__ unsigned g_attn_err;

struct AttnArgs {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int n_seqs, n_tokens, max_pages, max_q_len, max_kv_len;
  const uint32_t* codes[2];
  const uint16_t* scales[2];
  int n_kv_heads, page_size, n_pages, group;  // group: query heads of a KV head
  exq_rows q, out;
  int n_heads;
  float scale_log2;  // scale * log2(e)
  int causal, window;
  float* lse;
};

template <int VPL, int B>
__device__ __forceinline__ void load_group(const uint32_t* codes, const uint16_t* scales, long long g, int lane,
                                           float (&x)[VPL]) {
  constexpr int D = 32 * VPL;
  if constexpr (B == 16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(codes) + g * D + lane * VPL;
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = half_bits_to_float(__ldg(p + i));
  } else {
    const uint32_t* w = codes + g * (D * B / 32);
    const float s = half_bits_to_float(__ldg(scales + g));
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int bit = (lane * VPL + i) * B;
      const uint32_t lo = __ldg(w + (bit >> 5));
      const uint32_t hi = (bit & 31) + B > 32 ? __ldg(w + (bit >> 5) + 1) : 0u;
      const int u = static_cast<int>(fshr(lo, hi, bit & 31) & ((1u << B) - 1u));
      x[i] = static_cast<float>(u - (1 << (B - 1))) * s;
    }
  }
}

template <int VPL, int B>
__global__ void __launch_bounds__(128) attn_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int D = 32 * VPL;
  __shared__ float sm[4], sl[4], so[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x, h = blockIdx.y;
  int n = 0;
  for (int b = lane; b < a.n_seqs; b += 32) n += __ldg(a.q_start + b) <= t ? 1 : 0;
  const int b = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n))) - 1;
  if (t >= __ldg(a.q_start + a.n_seqs)) return;  // padding
  const int first = b >= 0 ? __ldg(a.q_start + b) : 0, next = b >= 0 ? __ldg(a.q_start + b + 1) : 0;
  const int len = b >= 0 ? __ldg(a.kv_len + b) : -1;
  if (next <= t || next - first > a.max_q_len || len < 0 || len > a.max_kv_len) {
    if (threadIdx.x == 0) atomicOr(&g_attn_err, kDevErrBadPage);
    return;
  }
  const int pos = len - (next - t);
  const int end = a.causal ? pos + 1 : len;
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const uint16_t* qp = a.q.data + t * a.q.token_stride + h * a.q.head_stride + lane * VPL;
  float q[VPL], o[VPL], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    q[i] = half_bits_to_float(qp[i]);
    o[i] = 0.f;
  }
  for (int j = begin + warp; j < end; j += 4) {
    const int page = __ldg(a.page_table + static_cast<long long>(b) * a.max_pages + j / a.page_size);
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) atomicOr(&g_attn_err, kDevErrBadPage);
      continue;
    }
    const long long g = (static_cast<long long>(page) * a.n_kv_heads + h / a.group) * a.page_size + j % a.page_size;
    float x[VPL], s = 0.f;
    load_group<VPL, B>(a.codes[0], a.scales[0], g, lane, x);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s += q[i] * x[i];
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= a.scale_log2;
    const float m1 = fmaxf(m, s), f = exp2f(m - m1), w = exp2f(s - m1);
    load_group<VPL, B>(a.codes[1], a.scales[1], g, lane, x);
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = o[i] * f + w * x[i];
    l = l * f + w;
    m = m1;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) so[warp][lane * VPL + i] = o[i];
  __syncthreads();
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float f[4], total = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = sl[w] > 0.f ? exp2f(sm[w] - mm) : 0.f;
    total += sl[w] * f[w];
  }
  uint16_t* out = a.out.data + t * a.out.token_stride + h * a.out.head_stride;
  for (int d = threadIdx.x; d < D; d += 128) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) y += so[w][d] * f[w];
    out[d] = static_cast<uint16_t>(float_to_half_bits(total > 0.f ? y / total : 0.f));
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[static_cast<long long>(t) * a.n_heads + h] = total > 0.f ? (mm + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

template <int VPL>
void (*attn_for_bits(int b))(const AttnArgs) {
  return b == 4 ? attn_kernel<VPL, 4> : b == 6 ? attn_kernel<VPL, 6> : b == 8 ? attn_kernel<VPL, 8> : attn_kernel<VPL, 16>;
}

constexpr size_t kCounterBytes = 64 << 10;  // the zero-filled start of the workspace

}  // namespace

size_t paged_attn_workspace_bytes(const exq_kv_cache&, const exq_kv_batch&, int, int) { return kCounterBytes; }

exq_status launch_paged_attn(const AttnCall& call, int, cudaStream_t stream) {
  const exq_kv_cache& c = *call.cache;
  const exq_kv_batch& b = *call.batch;
  AttnArgs a{};
  a.q_start = b.q_start;
  a.kv_len = b.kv_len;
  a.page_table = b.page_table;
  a.n_seqs = b.n_seqs;
  a.n_tokens = b.n_tokens;
  a.max_pages = b.max_pages;
  a.max_q_len = b.max_q_len;
  a.max_kv_len = b.max_kv_len;
  const long long groups = static_cast<long long>(c.n_pages) * c.n_kv_heads * c.page_size * call.layer;
  a.codes[0] = c.k_codes + groups * (c.D * c.bits / 32);
  a.codes[1] = c.v_codes + groups * (c.D * c.bits / 32);
  if (c.bits != 16) {
    a.scales[0] = c.k_scales + groups;
    a.scales[1] = c.v_scales + groups;
  }
  a.n_kv_heads = c.n_kv_heads;
  a.page_size = c.page_size;
  a.n_pages = c.n_pages;
  a.group = call.n_heads / c.n_kv_heads;
  a.q = call.q;
  a.out = call.out;
  a.n_heads = call.n_heads;
  a.scale_log2 = static_cast<float>(call.scale * 1.4426950408889634);
  a.causal = call.causal;
  a.window = call.window;
  a.lse = call.lse;
  auto fn = c.D == 64 ? attn_for_bits<2>(c.bits) : c.D == 128 ? attn_for_bits<4>(c.bits) : attn_for_bits<8>(c.bits);
  fn<<<dim3(b.n_tokens, call.n_heads), 128, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

unsigned take_attn_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_attn_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_attn_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
