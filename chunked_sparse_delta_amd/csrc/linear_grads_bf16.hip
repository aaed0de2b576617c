// Linear attention, the gradients of q, k and v: bfloat16 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_grads_bf16(const AttendArgs &a, hipStream_t st) { return attend_grads<bf16>(a, st); }
hipError_t grads_prepare_bf16() { return grads_prepare<bf16>(); }

}  // namespace sdm
