// Layer norm, forward, from a float32 X (layer_norm_fwd.cuh).
#include "layer_norm_fwd.cuh"

namespace metis {

void norm_fwd_f32(const NormFwdParams& p, int mode, bool save, int num_sms, cudaStream_t s) {
  using T = float;
  if (mode == kAny)
    norm_fwd_cols<T, 1, kAny, false>(p, num_sms, s);
  else if (mode == kPhase)
    norm_fwd_cols<T, 4, kPhase, false>(p, num_sms, s);
  else
    save ? norm_fwd_cols<T, 4, kAligned, true>(p, num_sms, s) : norm_fwd_cols<T, 4, kAligned, false>(p, num_sms, s);
}

}  // namespace metis
