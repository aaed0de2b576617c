// Linear attention, the gradients of q, k and v: float32 rows.
#include "linear_attend.h"

namespace sdm {

hipError_t attend_grads_f32(const AttendArgs &a, hipStream_t st) { return attend_grads<float>(a, st); }
hipError_t grads_prepare_f32() { return grads_prepare<float>(); }

}  // namespace sdm
