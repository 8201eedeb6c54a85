// The few-row attention kernels of Q4 pages (one translation unit per format: they compile side by side).
#include "exq_attn_split.cuh"

namespace exq {

exq_status launch_attn_split4(const AttnCall& c, const AttnArgs& a, int unit_rows, int sms, cudaStream_t stream) {
  return split::launch_bits<4>(c, a, unit_rows, sms, stream);
}

}  // namespace exq
