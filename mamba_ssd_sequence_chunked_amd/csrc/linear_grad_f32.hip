// linear_grad_f32.hip - the walk's kernels for fp32 inputs, with the derivative for the decay.
#include "linear_dispatch.hpp"

namespace ssd {

template hipError_t launch_linear_walk<float, true, true>(const LinearWalk<float>&, hipStream_t);
template hipError_t launch_linear_walk<float, false, true>(const LinearWalk<float>&, hipStream_t);

}  // namespace ssd
