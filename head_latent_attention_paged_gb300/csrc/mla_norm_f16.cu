// The RMS norm's kernels for f16 rows.
#include "mla_norm.cuh"

namespace mla {
template cudaError_t launch_norm_of<__half>(const NormParams& p, cudaStream_t stream);
}  // namespace mla
