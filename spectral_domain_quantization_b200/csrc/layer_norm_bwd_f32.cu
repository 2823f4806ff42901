// Layer norm, backward, from a float32 X (layer_norm_bwd.cuh).
#include "layer_norm_bwd.cuh"

namespace metis {

int norm_bwd_f32(const NormBwdParams& p, int mode, bool narrow, int parts, bool occupancy, int num_sms, cudaStream_t s) {
  return norm_bwd_kind<float>(p, mode, narrow, parts, occupancy, num_sms, s);
}

}  // namespace metis
