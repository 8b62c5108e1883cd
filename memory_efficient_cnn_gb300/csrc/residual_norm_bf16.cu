// The residual norm's kernels in bf16.
#include "residual_norm_kernels.cuh"

namespace im2win {
namespace rnorm {
template cudaError_t launch_norm_forward<bf16_t>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<bf16_t>(const NormArgs &, const ColumnGrads &, void *, cudaStream_t);
}  // namespace rnorm
}  // namespace im2win
