// Paged decode attention: 4-bit cache, head dim 128.
#include "paged_decode.cuh"

namespace fl {

FL_DEFINE_PAGED(e2m1_d128, KV_E2M1, 128)

}  // namespace fl
