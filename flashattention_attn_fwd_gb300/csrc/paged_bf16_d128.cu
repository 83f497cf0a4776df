// Paged decode attention: bf16 cache, head dim 128.
#include "paged_decode.cuh"

namespace fl {

FL_DEFINE_PAGED(bf16_d128, KV_BF16, 128)

}  // namespace fl
