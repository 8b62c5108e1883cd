// The residual norm's kernels in f16.
#include "residual_norm_kernels.cuh"

namespace im2win {
namespace rnorm {
template cudaError_t launch_norm_forward<f16_t>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<f16_t>(const NormArgs &, const ColumnGrads &, void *, cudaStream_t);
}  // namespace rnorm
}  // namespace im2win
