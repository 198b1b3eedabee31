// linear_loss_bf16.hip -- linear_loss.h for bfloat16.
#include "linear_loss.h"

namespace tt {
template <> void linear_loss<__bf16>(const Call &c, const Sizes &z, uint8_t *ws, hipStream_t s) { enqueue<__bf16>(c, z, ws, s); }
}  // namespace tt
