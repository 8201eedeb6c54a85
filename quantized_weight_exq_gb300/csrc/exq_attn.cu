// Attention of new tokens over a paged (quantised) KV cache: the launch.
//   o = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q . k_t - m),
// over the cached tokens t a row sees, m the running maximum.
#include "exq_attn_chunk.cuh"

namespace exq {
namespace {

__device__ unsigned g_attn_err;

// its device address, looked up once per device
unsigned* error_word(int dev) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static unsigned* ptr[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_attn_err) == cudaSuccess)
      ptr[dev] = static_cast<unsigned*>(p);
    else
      cudaGetLastError();
  }
  return ptr[dev];
}

constexpr int kWaitLimit = 1 << 22;  // try_wait rounds before giving up

// Sequences of more query rows a KV head than these go to the tensor-memory
// kernel, whose units have 256 (128) of them; those of fewer to the
// packed-code kernel, which reads the cache again for every 16 (8). Measured
// on 8 sequences of up to 4000 tokens, packed-code against tensor-memory
// kernel, us: D = 128, Q4: 31 / 39 at 32 rows, 42 / 42 at 40, 45 / 40 at 64;
// fp16: 63 / 35 at 32; D = 64, Q4: 22 / 27 at 64; D = 256, Q4: 40 / 36 at 32.
int few_rows(const exq_kv_cache& c) { return c.bits == 16 || c.D == 256 ? 16 : c.D == 64 ? 64 : 32; }

// The launches of a call, by the host's bounds.
struct Plan {
  long long rows;             // rows a KV head of one sequence at most
  int few;                    // the limit of the packed-code kernel
  bool split, chunk;
  int split_rows, chunk_rows; // rows of their units
};

Plan plan_of(const exq_kv_cache& c, const exq_kv_batch& b, int n_heads) {
  const int group = n_heads / c.n_kv_heads;
  Plan p{};
  p.rows = static_cast<long long>(std::min(b.max_q_len, b.n_tokens)) * group;
  p.few = few_rows(c);
  p.chunk = p.rows > p.few;
  // Sequences of both kinds, as far as the host can tell: each launch passes
  // over the other's. A chunk of 2048 tokens with 63 single tokens over 4000
  // cached (Q4, 8 KV heads): 267 us, 423 with all of them in the
  // tensor-memory kernel; with 31 of 32 KV heads: 225 us, 583. Prompts of mixed
  // lengths pay 4 us for the second launch.
  const bool mixed = p.chunk && b.n_tokens < static_cast<long long>(b.n_seqs) * b.max_q_len && b.n_seqs > 1;
  p.split = !p.chunk || mixed;
  // beside prompt chunks the short sequences are mostly single tokens (units
  // of 16 rows there: 305 and 298 us)
  p.split_rows = split::rows_of(c.D, mixed ? group : p.rows);
  p.chunk_rows = chunk::rows_of(c.D);
  return p;
}

}  // namespace

size_t paged_attn_workspace_bytes(const exq_kv_cache& c, const exq_kv_batch& b, int n_heads, int sms) {
  const Plan p = plan_of(c, b, n_heads);
  const size_t split = p.split ? static_cast<size_t>(std::min(4 * sms, kAttnMaxCtas)) * p.split_rows : 0;
  const size_t chunk = p.chunk ? static_cast<size_t>(std::min(sms, kAttnMaxCtas)) * p.chunk_rows : 0;
  return kAttnCounterBytes + std::max(split, chunk) * 2 * (c.D + 2) * sizeof(float);
}

exq_status launch_paged_attn(const AttnCall& call, int sms, cudaStream_t stream) {
  const exq_kv_cache& c = *call.cache;
  const exq_kv_batch& b = *call.batch;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return EXQ_ERR_CUDA;
  AttnArgs a{};
  a.err = error_word(dev);
  if (!a.err) return EXQ_ERR_CUDA;
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
  a.window = call.window < b.max_kv_len ? call.window : 0;  // no position reaches that far: no limit, no overflow
  a.lse = call.lse;
  a.counters = static_cast<unsigned*>(call.workspace);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(call.workspace) + kAttnCounterBytes);
  const int starve = testing_starve_rounds();
  a.wait_limit = starve > 0 ? starve : kWaitLimit;
  a.starve = starve > 0 ? 1 : 0;
  const Plan plan = plan_of(c, b, call.n_heads);
  if (plan.rows > 0x7FFFFF00ll || plan.rows / 8 * b.n_seqs > 0x7FFFFF00ll)
    return EXQ_ERR_UNSUPPORTED;  // row and block numbers have 32 bits
  a.min_tiles = 2;  // 10 us for one sequence of 500 tokens, 15 at ten
  // What a unit's queries, joins and stores take, in tiles. Packed-code kernel,
  // us at 3, 6 and 12: 32 ragged sequences Q4 48, 44, 46 (61 at 0); 16 of 4000,
  // 32 KV heads 48, 47, 49; 40 of 3000, D = 64 Q8 19, 18, 18; 24 of 5000 fp16 62,
  // 56, 56. Tensor-memory kernel at 6, 12 and 24: prompts of 3500 in a window
  // 233, 230, 239 (360 at 0); 4 of 3000, D = 64 Q8 88, 86, 97; 3 of 900 Q4 84, 85, 81.
  if (plan.chunk) {
    a.rows_above = plan.split ? plan.few : 0;
    a.rows_upto = static_cast<int>(plan.rows);
    a.row_blocks = static_cast<int>((plan.rows + plan.chunk_rows - 1) / plan.chunk_rows);
    a.unit_cost = 12;
    const exq_status st = c.bits == 4   ? launch_attn_chunk4(call, a, sms, stream)
                          : c.bits == 6 ? launch_attn_chunk6(call, a, sms, stream)
                          : c.bits == 8 ? launch_attn_chunk8(call, a, sms, stream)
                                        : launch_attn_chunk16(call, a, sms, stream);
    if (st != EXQ_OK || !plan.split) return st;
  }
  a.rows_above = 0;
  a.rows_upto = static_cast<int>(std::min<long long>(plan.rows, plan.few));
  a.row_blocks = (a.rows_upto + plan.split_rows - 1) / plan.split_rows;
  a.unit_cost = 6;
  if (a.row_blocks == 0) return EXQ_OK;
  switch (c.bits) {
    case 4: return launch_attn_split4(call, a, plan.split_rows, sms, stream);
    case 6: return launch_attn_split6(call, a, plan.split_rows, sms, stream);
    case 8: return launch_attn_split8(call, a, plan.split_rows, sms, stream);
    default: return launch_attn_split16(call, a, plan.split_rows, sms, stream);
  }
}

unsigned take_attn_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_attn_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_attn_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
