// Linear attention, the gradients of q and k: float32 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_keys_f32(const AttendArgs &a, hipStream_t st) { return attend<float, true>(a, nullptr, st); }
hipError_t attend_prepare_keys_f32() { return attend_prepare<float, true>(); }

}  // namespace sdm
