// Attention of chunks over a bf16 paged cache, head dim 128.
#include "paged_prefill.cuh"

namespace fl {
cudaError_t launch_prefill_bf16_d128(int score_mod, const CUtensorMap* maps, const PrefillParams& p, cudaStream_t s) {
  return launch_prefill<KV_BF16, 128>(score_mod, maps, p, s);
}
}  // namespace fl
