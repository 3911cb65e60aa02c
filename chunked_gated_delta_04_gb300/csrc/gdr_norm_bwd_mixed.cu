// gdr_norm_bwd_mixed.cu -- the block norms' backward for bf16 activations and fp32 residuals.
#include "gdr_norm_bwd.cuh"

namespace gdr {
template cudaError_t norm_bwd_launch<__nv_bfloat16, float>(const NormDims&, const NormBwdPtrs&, int, long long*, cudaStream_t);
}  // namespace gdr
