// Linear attention, the readings and the gradient of v: float32 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_values_f32(const AttendArgs &a, const StateArgs *single, hipStream_t st) { return attend<float, false>(a, single, st); }
hipError_t attend_prepare_values_f32() { return attend_prepare<float, false>(); }

}  // namespace sdm
