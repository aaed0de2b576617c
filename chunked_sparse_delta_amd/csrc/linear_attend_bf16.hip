// Linear attention, the readings: bfloat16 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_bf16(const AttendArgs &a, const StateArgs *single, hipStream_t st) { return attend<bf16>(a, single, st); }
hipError_t attend_prepare_bf16() { return attend_prepare<bf16>(); }

}  // namespace sdm
