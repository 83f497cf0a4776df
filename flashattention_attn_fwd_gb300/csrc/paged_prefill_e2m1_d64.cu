// Attention of chunks over a 4-bit paged cache, head dim 64.
#include "paged_prefill.cuh"

namespace fl {
cudaError_t launch_prefill_e2m1_d64(int score_mod, const CUtensorMap* maps, const PrefillParams& p, cudaStream_t s) {
  return launch_prefill<KV_E2M1, 64>(score_mod, maps, p, s);
}
}  // namespace fl
