// Layer norm, backward, from a float32 X (layer_norm_bwd.cuh).
#include "layer_norm_bwd.cuh"

namespace metis {

int norm_bwd_f32(const NormBwdParams& p, int parts, bool occupancy, cudaStream_t s) {
  return norm_bwd_kind<float>(p, parts, occupancy, s);
}

}  // namespace metis
