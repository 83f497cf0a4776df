// Paged decode attention: 4-bit cache, head dim 64.
#include "paged_decode.cuh"

namespace fl {

FL_DEFINE_PAGED(e2m1_d64, KV_E2M1, 64)

}  // namespace fl
