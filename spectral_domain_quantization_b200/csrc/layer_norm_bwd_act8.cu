// Layer norm, backward, from a 8-bit X (layer_norm_bwd.cuh).
#include "layer_norm_bwd.cuh"

namespace metis {

int norm_bwd_act8(const NormBwdParams& p, int parts, bool occupancy, cudaStream_t s) {
  return norm_bwd_kind<Act8Tag>(p, parts, occupancy, s);
}

}  // namespace metis
