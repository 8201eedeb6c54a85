// Host entry points of libexq: argument checks, dispatch, status codes.
// Every check here runs before any launch and has no side effects.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "exq_internal.h"
#include "exq_testing.h"

namespace exq {

const DeviceInfo& device_info(int device) {
  constexpr int kMaxDevices = 64;
  static DeviceInfo infos[kMaxDevices];
  static std::once_flag once[kMaxDevices];
  static DeviceInfo none;
  if (device < 0 || device >= kMaxDevices) return none;
  std::call_once(once[device], [device] {
    DeviceInfo d;
    cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, device);
    cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
    cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, device);
    cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, device);
    infos[device] = d;
  });
  return infos[device];
}

EncodeTiled tensor_map_encoder() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer,
               uint64_t outer_stride_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapL2promotion promotion) {
  EncodeTiled enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t gdim[2] = {inner, outer};
  const cuuint64_t gstride[1] = {outer_stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t es[2] = {1, 1};
  return enc(map, type, 2, const_cast<void*>(base), gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, promotion,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {
std::atomic<int> g_starve_rounds{0};
}  // namespace

int testing_starve_rounds() { return g_starve_rounds.load(std::memory_order_relaxed); }

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// structural checks of a layer descriptor (host-visible fields only)
exq_status check_weight(const exq_weight* w) {
  if (!w) return EXQ_ERR_INVALID_ARG;
  if (w->K <= 0 || w->N <= 0 || w->N % 8 || w->K % 32) return EXQ_ERR_INVALID_ARG;
  if (!w->qweight || !aligned16(w->qweight)) return EXQ_ERR_INVALID_ARG;
  if (w->perm && !aligned16(w->perm)) return EXQ_ERR_INVALID_ARG;
  // fp16 scales, or (EXL2 two-level) codes and column maxima instead
  const bool two_level = w->format == EXQ_FMT_EXL2_QSCALE;
  if (two_level) {
    if (w->scales || !w->q_scale || !w->q_scale_max || !aligned16(w->q_scale) || !aligned16(w->q_scale_max))
      return EXQ_ERR_INVALID_ARG;
  } else {
    if (!w->scales || !aligned16(w->scales) || w->q_scale || w->q_scale_max) return EXQ_ERR_INVALID_ARG;
  }
  if (w->format == EXQ_FMT_GPTQ4) {
    if (w->group_size <= 0 || w->group_size % 32 || w->K % w->group_size) return EXQ_ERR_INVALID_ARG;
    if (w->n_groups != w->K / w->group_size || w->n_word_rows != w->K / 8) return EXQ_ERR_INVALID_ARG;
    if (!w->qzeros || !aligned16(w->qzeros) || w->seg_word_off) return EXQ_ERR_INVALID_ARG;
  } else if (w->format == EXQ_FMT_EXL2 || two_level) {
    if (w->group_size != 32 || w->n_groups != w->K / 32) return EXQ_ERR_INVALID_ARG;
    if (w->n_word_rows < 2 * w->n_groups || w->n_word_rows > 8 * w->n_groups) return EXQ_ERR_INVALID_ARG;
    if (!w->seg_word_off || w->qzeros) return EXQ_ERR_INVALID_ARG;
  } else {
    return EXQ_ERR_INVALID_ARG;
  }
  return EXQ_OK;
}

// layers of one exq_gemv_multi call: each valid, one format, one K, one group size
exq_status check_group(const exq_weight* w, int n) {
  if (!w || n < 1 || n > EXQ_GEMV_MAX_LAYERS) return EXQ_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const exq_status st = check_weight(&w[i]);
    if (st != EXQ_OK) return st;
    if (w[i].format != w[0].format || w[i].K != w[0].K || w[i].group_size != w[0].group_size)
      return EXQ_ERR_INVALID_ARG;
  }
  return EXQ_OK;
}

int current_cc() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const DeviceInfo& di = device_info(dev);
  return di.cc_major * 10 + di.cc_minor;
}

}  // namespace
}  // namespace exq

using namespace exq;

extern "C" exq_status exq_dequant(const exq_weight* w, uint16_t* W_out, void* stream) {
  const exq_status st = check_weight(w);
  if (st != EXQ_OK) return st;
  if (!W_out || !aligned16(W_out)) return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_dequant(*w, W_out, static_cast<cudaStream_t>(stream));
}

extern "C" size_t exq_gemv_workspace_size(const exq_weight* w, int32_t M) {
  if (check_weight(w) != EXQ_OK || M < 1 || M > 16) return 0;
  return gemv_workspace_bytes(w, 1, M);
}

extern "C" exq_status exq_gemv(const exq_weight* w, const uint16_t* x, int32_t M, uint16_t* y, void* workspace,
                               size_t ws_bytes, void* stream) {
  const exq_status st = check_weight(w);
  if (st != EXQ_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y) || M < 1) return EXQ_ERR_INVALID_ARG;
  if (M > 16) return EXQ_ERR_UNSUPPORTED;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_gemv(w, 1, x, M, &y, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" size_t exq_gemv_multi_workspace_size(const exq_weight* w, int32_t n, int32_t M) {
  if (check_group(w, n) != EXQ_OK || M < 1 || M > 16) return 0;
  return gemv_workspace_bytes(w, n, M);
}

extern "C" exq_status exq_gemv_multi(const exq_weight* w, int32_t n, const uint16_t* x, int32_t M,
                                     uint16_t* const* y, void* workspace, size_t ws_bytes, void* stream) {
  const exq_status st = check_group(w, n);
  if (st != EXQ_OK) return st;
  if (!x || !y || !aligned16(x) || M < 1) return EXQ_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!y[i] || !aligned16(y[i])) return EXQ_ERR_INVALID_ARG;
  if (M > 16) return EXQ_ERR_UNSUPPORTED;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_gemv(w, n, x, M, y, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" size_t exq_gemm_workspace_size(const exq_weight* w, int32_t M) {
  if (check_weight(w) != EXQ_OK || M < 1) return 0;
  return gemm_workspace_bytes(w, 1, M);
}

extern "C" size_t exq_gemm_multi_workspace_size(const exq_weight* w, int32_t n, int32_t M) {
  if (n > EXQ_GEMM_MAX_LAYERS || check_group(w, n) != EXQ_OK || M < 1) return 0;
  return gemm_workspace_bytes(w, n, M);
}

extern "C" exq_status exq_gemm_multi(const exq_weight* w, int32_t n, const uint16_t* x, int32_t M,
                                     uint16_t* const* y, void* workspace, size_t ws_bytes, void* stream) {
  if (n > EXQ_GEMM_MAX_LAYERS) return EXQ_ERR_INVALID_ARG;
  const exq_status st = check_group(w, n);
  if (st != EXQ_OK) return st;
  if (!x || !y || !aligned16(x) || M < 1) return EXQ_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (!y[i] || !aligned16(y[i])) return EXQ_ERR_INVALID_ARG;
    if (w[i].K % 64 || w[i].N % 128) return EXQ_ERR_UNSUPPORTED;
  }
  const size_t need = gemm_workspace_bytes(w, n, M);
  if (need && (!workspace || ws_bytes < need || !aligned16(workspace))) return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_gemm(w, n, x, M, y, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" exq_status exq_gemm(const exq_weight* w, const uint16_t* x, int32_t M, uint16_t* y, void* workspace,
                               size_t ws_bytes, void* stream) {
  const exq_status st = check_weight(w);
  if (st != EXQ_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y) || M < 1) return EXQ_ERR_INVALID_ARG;
  const size_t need = gemm_workspace_bytes(w, 1, M);
  if (need && (!workspace || ws_bytes < need || !aligned16(workspace))) return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_gemm(w, 1, x, M, &y, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" exq_status exq_gemm_noalloc(const exq_weight* w, const uint16_t* x, int32_t M, uint16_t* y,
                                       void* stream) {
  const exq_status st = check_weight(w);
  if (st != EXQ_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y) || M < 1) return EXQ_ERR_INVALID_ARG;
  if (gemm_gather_bytes(*w, M) > EXQ_NOALLOC_SCRATCH_BYTES) return EXQ_ERR_UNSUPPORTED;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_gemm_noalloc(*w, x, M, y, static_cast<cudaStream_t>(stream));
}

namespace {
// EXQ_OK with `empty` set: nothing to do (n_groups == 0; the pointers are not used)
exq_status check_kv(const void* a, const void* b, const void* c, long long n_groups, int D, int bits, bool& empty) {
  if (n_groups < 0) return EXQ_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 256) || (bits != 4 && bits != 6 && bits != 8)) return EXQ_ERR_UNSUPPORTED;
  empty = n_groups == 0;
  if (empty) return EXQ_OK;
  if (!a || !b || !c || !aligned16(a) || !aligned16(b) || !aligned16(c)) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}
}  // namespace

extern "C" exq_status exq_kv_quantize(const uint16_t* x, int64_t n_groups, int32_t D, int32_t bits, uint32_t* codes,
                                      uint16_t* scales, void* stream) {
  bool empty = false;
  const exq_status st = check_kv(x, codes, scales, n_groups, D, bits, empty);
  if (st != EXQ_OK || empty) return st;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_kv_quantize(x, n_groups, D, bits, codes, scales, static_cast<cudaStream_t>(stream));
}

extern "C" exq_status exq_kv_dequantize(const uint32_t* codes, const uint16_t* scales, int64_t n_groups, int32_t D,
                                        int32_t bits, uint16_t* x_out, void* stream) {
  bool empty = false;
  const exq_status st = check_kv(codes, scales, x_out, n_groups, D, bits, empty);
  if (st != EXQ_OK || empty) return st;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_kv_dequantize(codes, scales, n_groups, D, bits, x_out, static_cast<cudaStream_t>(stream));
}

namespace {
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

exq_status check_rows(const exq_rows* r) {
  if (!r || !r->data || !aligned16(r->data) || r->token_stride % 8 || r->head_stride % 8) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}

// rows that are overwritten by a call that reads `in`: in's own rows, or other ones
exq_status check_in_place(const exq_rows& in, const exq_rows& out) {
  if (in.data == out.data && (in.token_stride != out.token_stride || in.head_stride != out.head_stride))
    return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}

exq_status check_rope(const exq_rope_params* r, int D) {
  if (!r || !r->steps || (reinterpret_cast<uintptr_t>(r->steps) & 7u) || r->R < 2 || r->R % 2 || r->R > D)
    return EXQ_ERR_INVALID_ARG;
  if (r->layout != EXQ_ROPE_HALF && r->layout != EXQ_ROPE_INTERLEAVED) return EXQ_ERR_INVALID_ARG;
  if (!std::isfinite(r->gain)) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}

exq_status check_cache(const exq_kv_cache* c) {
  if (!c || c->n_kv_heads <= 0 || c->n_pages <= 0 || c->n_layers <= 0) return EXQ_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128 && c->D != 256) return EXQ_ERR_UNSUPPORTED;
  if (c->bits != 4 && c->bits != 6 && c->bits != 8 && c->bits != 16) return EXQ_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return EXQ_ERR_UNSUPPORTED;
  if (c->n_kv_heads > 1024) return EXQ_ERR_UNSUPPORTED;
  if (!c->k_codes || !c->v_codes || !aligned16(c->k_codes) || !aligned16(c->v_codes)) return EXQ_ERR_INVALID_ARG;
  if (c->bits == 16) return c->k_scales || c->v_scales ? EXQ_ERR_INVALID_ARG : EXQ_OK;
  if (!c->k_scales || !c->v_scales || !aligned16(c->k_scales) || !aligned16(c->v_scales)) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}

exq_status check_batch(const exq_kv_cache& c, const exq_kv_batch* b) {
  if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_q_len < 0 || b->max_kv_len < 0 || b->max_pages < 0)
    return EXQ_ERR_INVALID_ARG;
  if (b->max_kv_len > static_cast<long long>(b->max_pages) * c.page_size) return EXQ_ERR_INVALID_ARG;
  if (b->n_seqs == 0 || b->n_tokens == 0) return EXQ_OK;  // nothing to do, the arrays are not looked at
  if (!b->q_start || !b->kv_len || !aligned4(b->q_start) || !aligned4(b->kv_len)) return EXQ_ERR_INVALID_ARG;
  if (b->max_pages > 0 && (!b->page_table || !aligned4(b->page_table))) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}

int current_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return device_info(dev).sm_count;
}
}  // namespace

extern "C" exq_status exq_rope(const exq_rope_params* rope, const exq_rows* x, int64_t n_tokens, int32_t n_heads,
                               int32_t D, const int32_t* pos, const exq_rows* y, int32_t grad, void* stream) {
  if (n_tokens < 0 || n_heads < 0 || D <= 0 || (grad != 0 && grad != 1)) return EXQ_ERR_INVALID_ARG;
  if (D % 8 || D > 512) return EXQ_ERR_UNSUPPORTED;
  exq_status st = check_rope(rope, D);
  if (st != EXQ_OK) return st;
  if (n_tokens == 0 || n_heads == 0) return EXQ_OK;
  if ((st = check_rows(x)) != EXQ_OK || (st = check_rows(y)) != EXQ_OK || (st = check_in_place(*x, *y)) != EXQ_OK) return st;
  if (!pos || !aligned4(pos)) return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_rope(*rope, *x, n_tokens, n_heads, D, pos, *y, grad != 0, current_sms(), static_cast<cudaStream_t>(stream));
}

extern "C" exq_status exq_kv_append(const exq_kv_cache* cache, int32_t layer, const exq_kv_batch* batch,
                                    const exq_rows* k, const exq_rows* v, const exq_rope_params* rope,
                                    const int32_t* pos, const exq_rows* q, const exq_rows* q_out, int32_t n_heads,
                                    void* stream) {
  exq_status st = check_cache(cache);
  if (st != EXQ_OK || (st = check_batch(*cache, batch)) != EXQ_OK) return st;
  if (layer < 0 || layer >= cache->n_layers) return EXQ_ERR_INVALID_ARG;
  if (rope ? (st = check_rope(rope, cache->D)) != EXQ_OK : pos != nullptr) return EXQ_ERR_INVALID_ARG;
  if (!aligned4(pos) || (q == nullptr) != (q_out == nullptr) || (q && (!rope || n_heads <= 0))) return EXQ_ERR_INVALID_ARG;
  if (batch->n_tokens == 0 || batch->n_seqs == 0) return EXQ_OK;
  if ((st = check_rows(k)) != EXQ_OK || (st = check_rows(v)) != EXQ_OK) return st;
  if (q && ((st = check_rows(q)) != EXQ_OK || (st = check_rows(q_out)) != EXQ_OK ||
            (st = check_in_place(*q, *q_out)) != EXQ_OK))
    return st;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_kv_append(*cache, layer, *batch, *k, *v, rope, pos, q, q_out, n_heads, current_sms(),
                          static_cast<cudaStream_t>(stream));
}

namespace {
exq_status check_attn(const exq_kv_cache* cache, const exq_kv_batch* batch, int n_heads) {
  exq_status st = check_cache(cache);
  if (st != EXQ_OK || (st = check_batch(*cache, batch)) != EXQ_OK) return st;
  if (n_heads <= 0 || n_heads % cache->n_kv_heads) return EXQ_ERR_INVALID_ARG;
  if (n_heads > 4096) return EXQ_ERR_UNSUPPORTED;
  return EXQ_OK;
}
}  // namespace

extern "C" size_t exq_paged_attn_workspace_size(const exq_kv_cache* cache, const exq_kv_batch* batch, int32_t n_heads) {
  const int sms = current_sms();
  if (check_attn(cache, batch, n_heads) != EXQ_OK || sms <= 0) return 0;
  return paged_attn_workspace_bytes(*cache, *batch, n_heads, sms);
}

extern "C" exq_status exq_paged_attn(const exq_kv_cache* cache, int32_t layer, const exq_kv_batch* batch,
                                     const exq_rows* q, int32_t n_heads, float scale, int32_t causal, int32_t window,
                                     const exq_rows* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  exq_status st = check_attn(cache, batch, n_heads);
  if (st != EXQ_OK) return st;
  if (layer < 0 || layer >= cache->n_layers || !std::isfinite(scale) || (causal != 0 && causal != 1) || window < 0 ||
      !aligned4(lse))
    return EXQ_ERR_INVALID_ARG;
  if (batch->n_tokens == 0 || batch->n_seqs == 0) return EXQ_OK;
  if ((st = check_rows(q)) != EXQ_OK || (st = check_rows(out)) != EXQ_OK) return st;
  if (q->data == out->data) return EXQ_ERR_INVALID_ARG;
  const int sms = current_sms();
  if (sms <= 0 || current_cc() < 100) return EXQ_ERR_CUDA;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      ws_bytes < paged_attn_workspace_bytes(*cache, *batch, n_heads, sms))
    return EXQ_ERR_INVALID_ARG;
  const AttnCall call{cache, layer, batch, *q, *out, n_heads, scale, causal != 0, window, lse, workspace};
  return launch_paged_attn(call, sms, static_cast<cudaStream_t>(stream));
}

extern "C" exq_status exq_kv_copy_pages(const exq_kv_cache* cache, const int32_t* pairs, int64_t n_pairs, void* stream) {
  const exq_status st = check_cache(cache);
  if (st != EXQ_OK) return st;
  if (n_pairs < 0) return EXQ_ERR_INVALID_ARG;
  if (n_pairs == 0) return EXQ_OK;
  if (!pairs || !aligned4(pairs)) return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_kv_copy(*cache, pairs, n_pairs, current_sms(), static_cast<cudaStream_t>(stream));
}

namespace {
exq_status check_convert(const uint16_t* W, const int32_t* perm, int K, int N) {
  if (!W || !aligned16(W) || (perm && !aligned16(perm))) return EXQ_ERR_INVALID_ARG;
  if (K <= 0 || N <= 0 || K % 32 || N % 8) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}
}  // namespace

extern "C" exq_status exq_quantize_exl2(const uint16_t* W, const int32_t* perm, int32_t K, int32_t N,
                                        const uint32_t* seg_word_off, int32_t n_word_rows, uint32_t* qweight_out,
                                        uint16_t* scales_out, void* stream) {
  const exq_status st = check_convert(W, perm, K, N);
  if (st != EXQ_OK) return st;
  if (!seg_word_off || !qweight_out || !scales_out || !aligned16(seg_word_off) || !aligned16(qweight_out) ||
      !aligned16(scales_out))
    return EXQ_ERR_INVALID_ARG;
  if (n_word_rows < 2 * (K / 32) || n_word_rows > 8 * (K / 32)) return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_rtn_quantize(W, perm, K, N, seg_word_off, n_word_rows, qweight_out, scales_out,
                             static_cast<cudaStream_t>(stream));
}

extern "C" size_t exq_measure_exl2_workspace_size(int32_t K, int32_t N) {
  if (K <= 0 || N <= 0 || K % 32 || N % 8) return 0;
  return measure_workspace_bytes(K, N);
}

extern "C" exq_status exq_measure_exl2(const uint16_t* W, const int32_t* perm, int32_t K, int32_t N, float* err_out,
                                       void* workspace, size_t ws_bytes, void* stream) {
  const exq_status st = check_convert(W, perm, K, N);
  if (st != EXQ_OK) return st;
  if (!err_out || !aligned16(err_out) || !workspace || !aligned16(workspace) ||
      ws_bytes < measure_workspace_bytes(K, N))
    return EXQ_ERR_INVALID_ARG;
  if (current_cc() < 100) return EXQ_ERR_CUDA;
  return launch_rtn_measure(W, perm, K, N, err_out, workspace, static_cast<cudaStream_t>(stream));
}

extern "C" const char* exq_status_string(exq_status s) {
  switch (s) {
    case EXQ_OK: return "ok";
    case EXQ_ERR_INVALID_ARG: return "invalid argument";
    case EXQ_ERR_UNSUPPORTED: return "unsupported shape or format";
    case EXQ_ERR_CUDA: return "CUDA error";
    case EXQ_ERR_TIMEOUT: return "device wait timed out";
    case EXQ_ERR_FULL: return "no free page left";
  }
  return "unknown status";
}

extern "C" exq_status exq_get_last_device_error(void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned a = take_gemv_errors(s), b = take_dequant_errors(s), c = take_gemm_errors(s),
                 d = take_convert_errors(s), e = take_kv_errors(s), f = take_attn_errors(s);
  if (a == ~0u || b == ~0u || c == ~0u || d == ~0u || e == ~0u || f == ~0u) return EXQ_ERR_CUDA;
  const unsigned v = a | b | c | d | e | f;
  if (v & kDevErrTimeout) return EXQ_ERR_TIMEOUT;
  if (v & (kDevErrBadSegment | kDevErrBadPerm | kDevErrBadPage)) return EXQ_ERR_INVALID_ARG;
  return EXQ_OK;
}

extern "C" void exq_testing_starve(int32_t wait_rounds) {
  g_starve_rounds.store(wait_rounds > 0 ? wait_rounds : 0, std::memory_order_relaxed);
}
