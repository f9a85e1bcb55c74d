// linear_grad_bf16.hip - the walk's kernels for bf16 inputs, with the derivative for the decay.
#include "linear_dispatch.hpp"

namespace ssd {

template hipError_t launch_linear_walk<bf16, true, true>(const LinearWalk<bf16>&, hipStream_t);
template hipError_t launch_linear_walk<bf16, false, true>(const LinearWalk<bf16>&, hipStream_t);

}  // namespace ssd
