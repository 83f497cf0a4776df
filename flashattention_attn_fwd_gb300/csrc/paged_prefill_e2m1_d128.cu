// Attention of chunks over a 4-bit paged cache, head dim 128.
#include "paged_prefill.cuh"

namespace fl {
cudaError_t launch_prefill_e2m1_d128(int score_mod, const CUtensorMap* maps, const PrefillParams& p, cudaStream_t s) {
  return launch_prefill<KV_E2M1, 128>(score_mod, maps, p, s);
}
}  // namespace fl
