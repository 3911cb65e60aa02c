// gdr_norm_bwd_f32.cu -- the block norms' backward for fp32 activations and fp32 residuals.
#include "gdr_norm_bwd.cuh"

namespace gdr {
template cudaError_t norm_bwd_launch<float, float>(const NormDims&, const NormBwdPtrs&, int, long long*, cudaStream_t);
}  // namespace gdr
