// The residual norm's kernels in f32.
#include "residual_norm_kernels.cuh"

namespace im2win {
namespace rnorm {
template cudaError_t launch_norm_forward<float>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<float>(const NormArgs &, const ColumnGrads &, void *, cudaStream_t);
}  // namespace rnorm
}  // namespace im2win
