// The many-row attention kernels of Q4 pages (one translation unit per format: they compile side by side).
#include "exq_attn_chunk.cuh"

namespace exq {

exq_status launch_attn_chunk4(const AttnCall& c, const AttnArgs& a, int sms, cudaStream_t stream) {
  return chunk::launch_bits<4>(c, a, sms, stream);
}

}  // namespace exq
