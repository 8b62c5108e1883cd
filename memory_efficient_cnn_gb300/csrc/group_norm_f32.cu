// The group norm's kernels in f32.
#include "group_norm_kernels.cuh"

namespace im2win {
namespace gnorm {
template cudaError_t launch_forward<float>(const GroupArgs &, cudaStream_t);
template cudaError_t launch_backward<float>(const GroupArgs &, cudaStream_t);
}  // namespace gnorm
}  // namespace im2win
