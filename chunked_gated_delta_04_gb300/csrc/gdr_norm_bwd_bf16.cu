// gdr_norm_bwd_bf16.cu -- the block norms' backward for bf16 activations and bf16 residuals.
#include "gdr_norm_bwd.cuh"

namespace gdr {
template cudaError_t norm_bwd_launch<__nv_bfloat16, __nv_bfloat16>(const NormDims&, const NormBwdPtrs&, int, long long*, cudaStream_t);
}  // namespace gdr
