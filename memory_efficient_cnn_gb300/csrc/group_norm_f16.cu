// The group norm's kernels in f16.
#include "group_norm_kernels.cuh"

namespace im2win {
namespace gnorm {
template cudaError_t launch_forward<f16_t>(const GroupArgs &, cudaStream_t);
template cudaError_t launch_backward<f16_t>(const GroupArgs &, cudaStream_t);
}  // namespace gnorm
}  // namespace im2win
