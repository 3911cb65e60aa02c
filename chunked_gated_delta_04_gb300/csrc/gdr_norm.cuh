// gdr_norm.cuh -- row layout of the block norms' kernels (gdr_norm.cu, gdr_norm_bwd.cu).
//
// TPR threads hold a row of D channels in registers, K chunks of 8 channels each (chunk k of
// thread i: channels 8 (k TPR + i) ..).  Up to 32 threads share a warp and reduce by shuffles;
// more are a block of their own.
#pragma once

#include "gdr_block.cuh"

namespace gdr {

struct NormDims {
  long long rows;
  int heads, D;
  long long ld_x, ld_gate;  // token strides
  float eps;
  int vec;  // every pointer and stride 16-byte aligned and D a multiple of 8
};

template <typename IT>
__device__ __forceinline__ void load8(const IT* p, int c, int D, int vec, float (&v)[8]) {
  if (vec) {
    if (c < D) {
      load_v<8>(p + c, v);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < D ? to_f32(p[c + i]) : 0.f;
  }
}
template <typename IT>
__device__ __forceinline__ void store8(IT* p, int c, int D, int vec, const float (&v)[8]) {
  if (vec) {
    if (c < D) store_v<8>(p + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) p[c + i] = from_f32<IT>(v[i]);
  }
}

// Sums of M values over the TPR threads of a row, the same in each of them.  red: shared memory
// of 2 * M * TPR / 32 floats for TPR > 32, used in turns (flip) so that one barrier is enough.
template <int TPR, int M>
__device__ __forceinline__ void row_sums(float (&v)[M], float* red, int& flip) {
  constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = kIn / 2; o > 0; o >>= 1)
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    float* buf = red + flip * M * kWarps;
    flip ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int m = 0; m < M; ++m) buf[m * kWarps + warp] = v[m];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += buf[m * kWarps + w];
      v[m] = a;
    }
  }
}

// Threads per row and chunks per thread for a width: one chunk while a warp is enough, then blocks.
template <typename F>
cudaError_t norm_shape(int D, F f) {
#define GDR_NORM_SHAPE(tpr, k) \
  if (D <= 8 * (tpr) * (k)) return f(std::integral_constant<int, tpr>{}, std::integral_constant<int, k>{})
  GDR_NORM_SHAPE(8, 1);
  GDR_NORM_SHAPE(16, 1);
  GDR_NORM_SHAPE(32, 1);
  GDR_NORM_SHAPE(32, 2);
  GDR_NORM_SHAPE(128, 1);
  GDR_NORM_SHAPE(256, 1);
  GDR_NORM_SHAPE(512, 1);
  GDR_NORM_SHAPE(512, 2);
  GDR_NORM_SHAPE(512, 4);
#undef GDR_NORM_SHAPE
  return cudaErrorInvalidValue;
}
constexpr int kNormMaxD = 16384;

gdr_status resolve_norm(const gdr_norm_problem* p, NormDims* d);

}  // namespace gdr
