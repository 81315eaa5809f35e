// The sandwich norm's kernels for fp32.
#include "sandwich_kernels.h"

namespace monarch {

template hipError_t sandwich_launch_fwd<float>(const SandwichFwd&, hipStream_t);
template hipError_t sandwich_launch_bwd<float>(const SandwichBwd&, const SandwichBwdPlan&, hipStream_t);
template hipError_t sandwich_launch_join<float>(const SandwichJoin&, int64_t, hipStream_t);

}  // namespace monarch
