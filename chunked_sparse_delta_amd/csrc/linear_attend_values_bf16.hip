// Linear attention, the readings and the gradient of v: bfloat16 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_values_bf16(const AttendArgs &a, const StateArgs *single, hipStream_t st) { return attend<bf16, false>(a, single, st); }
hipError_t attend_prepare_values_bf16() { return attend_prepare<bf16, false>(); }

}  // namespace sdm
