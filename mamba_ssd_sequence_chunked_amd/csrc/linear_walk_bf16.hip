// linear_walk_bf16.hip - the walk's kernels for bf16 inputs.
#include "linear_dispatch.hpp"

namespace ssd {

template hipError_t launch_linear_walk<bf16, true, false>(const LinearWalk<bf16>&, hipStream_t);
template hipError_t launch_linear_walk<bf16, false, false>(const LinearWalk<bf16>&, hipStream_t);

}  // namespace ssd
