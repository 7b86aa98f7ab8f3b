// The RMS norm's kernels for f32 rows.
#include "mla_norm.cuh"

namespace mla {
template cudaError_t launch_norm_of<float>(const NormParams& p, cudaStream_t stream);
}  // namespace mla
