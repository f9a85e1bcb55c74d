// linear_walk_f32.hip - the walk's kernels for fp32 inputs.
#include "linear_dispatch.hpp"

namespace ssd {

template hipError_t launch_linear_walk<float, true, false>(const LinearWalk<float>&, hipStream_t);
template hipError_t launch_linear_walk<float, false, false>(const LinearWalk<float>&, hipStream_t);

}  // namespace ssd
