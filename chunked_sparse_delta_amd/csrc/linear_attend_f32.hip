// Linear attention, the readings: float32 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_f32(const AttendArgs &a, const StateArgs *single, hipStream_t st) { return attend<float>(a, single, st); }
hipError_t attend_prepare_f32() { return attend_prepare<float>(); }

}  // namespace sdm
