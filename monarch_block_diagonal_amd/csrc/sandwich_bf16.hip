// The sandwich norm's kernels for bfloat16.
#include "sandwich_kernels.h"

namespace monarch {

template hipError_t sandwich_launch_fwd<uint16_t>(const SandwichFwd&, hipStream_t);
template hipError_t sandwich_launch_bwd<uint16_t>(const SandwichBwd&, const SandwichBwdPlan&, hipStream_t);
template hipError_t sandwich_launch_join<uint16_t>(const SandwichJoin&, int64_t, hipStream_t);

}  // namespace monarch
