// The few-row attention kernels of Q6 pages (one translation unit per format: they compile side by side).
#include "exq_attn_split.cuh"

namespace exq {

exq_status launch_attn_split6(const AttnCall& c, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream) {
  return split::launch_bits<6>(c, a, unit_rows, sms, stream);
}

}  // namespace exq
