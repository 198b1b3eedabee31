// linear_loss_f16.hip -- linear_loss.h for float16.
#include "linear_loss.h"

namespace tt {
template <> void linear_loss<_Float16>(const Call &c, const Sizes &z, uint8_t *ws, hipStream_t s) { enqueue<_Float16>(c, z, ws, s); }
}  // namespace tt
