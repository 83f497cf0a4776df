// Paged decode attention: bf16 cache, head dim 64.
#include "paged_decode.cuh"

namespace fl {

FL_DEFINE_PAGED(bf16_d64, KV_BF16, 64)

}  // namespace fl
