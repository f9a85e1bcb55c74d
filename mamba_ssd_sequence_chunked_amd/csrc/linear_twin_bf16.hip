// linear_twin_bf16.hip - two walks in a launch for bf16 inputs.
#include "linear_dispatch.hpp"

namespace ssd {

template hipError_t launch_linear_twin<bf16, true>(const LinearWalk<bf16>&, const LinearWalk<bf16>&, hipStream_t);
template hipError_t launch_linear_twin<bf16, false>(const LinearWalk<bf16>&, const LinearWalk<bf16>&, hipStream_t);

}  // namespace ssd
