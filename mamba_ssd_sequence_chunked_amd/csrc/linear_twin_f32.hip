// linear_twin_f32.hip - two walks in a launch for fp32 inputs.
#include "linear_dispatch.hpp"

namespace ssd {

template hipError_t launch_linear_twin<float, true>(const LinearWalk<float>&, const LinearWalk<float>&, hipStream_t);
template hipError_t launch_linear_twin<float, false>(const LinearWalk<float>&, const LinearWalk<float>&, hipStream_t);

}  // namespace ssd
