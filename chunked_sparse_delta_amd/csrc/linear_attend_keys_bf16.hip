// Linear attention, the gradients of q and k: bfloat16 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_keys_bf16(const AttendArgs &a, hipStream_t st) { return attend<bf16, true>(a, nullptr, st); }
hipError_t attend_prepare_keys_bf16() { return attend_prepare<bf16, true>(); }

}  // namespace sdm
