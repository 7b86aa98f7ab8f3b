// The RMS norm's kernels for bf16 rows.
#include "mla_norm.cuh"

namespace mla {
template cudaError_t launch_norm_of<__nv_bfloat16>(const NormParams& p, cudaStream_t stream);
}  // namespace mla
