// gdr_norm.cuh -- row layout of the block norms' kernels (gdr_norm.cu, gdr_norm_bwd*.cu).
//
// TPR threads hold a row of D channels in registers, K chunks of 8 channels each: chunk k of thread i
// is channels 8 (k TPR + i) .., or, in the kernels for rows that do not take 16-byte accesses and fill
// a block (SIDE), channels (8 k + j) TPR + i for j < 8, so that a warp's single loads lie side by side.  Up to 32 threads share a warp and reduce by shuffles;
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

// The token of a row.  Rows that lie evenly apart (heads 1, to which the host brings what it can) take no
// division: with a 64-bit one per row, for eight channels a thread, gated 131072 x 128 took 61 us for both directions, now 58.6.
// (The staged rows of the backward, which have a block each, still take one.)
__device__ __forceinline__ long long token_of(const NormDims& d, long long row) {
  if (d.heads == 1) return row;
  return row < (1ll << 31) ? (long long)((uint32_t)row / (uint32_t)d.heads) : row / d.heads;
}

// Which tensors a call has.  The kernels are built for three combinations (norm_parts), where what is absent
// costs no registers, and once for any other (kNormAny: asked at run time).  A norm alone in front of a block, and one behind
// a scaled residual add, are among the others: 8192 x 4096, bf16, backward 78 us (bytes: 30) and 113 (60), where the
// residual add's own kernel takes 84 (50).
enum NormParts { kNormPost = 1, kNormGate = 2, kNormScale = 4, kNormPre = 8, kNormRes = 16, kNormAny = -1 };

// Eight neighbouring channels as they come from memory, converted where they are used, so that a
// load is not waited for before that.
template <typename IT>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
// Channel of element j of chunk k.
template <int TPR, bool SIDE>
__device__ __forceinline__ int channel(int k, int i0, int j) {
  return SIDE ? (8 * k + j) * TPR + i0 : 8 * (k * TPR + i0) + j;
}
// Chunk k of a row of D channels (zeros past its end); vec: in 16-byte accesses.
template <int TPR, bool SIDE, typename IT>
__device__ __forceinline__ Raw8<IT> load_raw8(const IT* p, int k, int i0, int D, int vec) {
  Raw8<IT> r;
  if (!SIDE && vec) {
    const int c = channel<TPR, SIDE>(k, i0, 0);
    if constexpr (sizeof(IT) == 4) {
      r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < D) {
        r.a = *reinterpret_cast<const float4*>(p + c);
        r.b = *reinterpret_cast<const float4*>(p + c + 4);
      }
    } else {
      r.w = make_uint4(0, 0, 0, 0);
      if (c < D) r.w = *reinterpret_cast<const uint4*>(p + c);
    }
  } else if constexpr (sizeof(IT) == 4) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = channel<TPR, SIDE>(k, i0, j) < D ? p[channel<TPR, SIDE>(k, i0, j)] : 0.f;
    r.a = make_float4(v[0], v[1], v[2], v[3]);
    r.b = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = channel<TPR, SIDE>(k, i0, j) < D ? q[channel<TPR, SIDE>(k, i0, j)] : 0;
    r.w = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  return r;
}
template <int TPR, bool SIDE, typename IT>
__device__ __forceinline__ void store8(IT* p, int k, int i0, int D, int vec, const float (&v)[8]) {
  if (!SIDE && vec) {
    const int c = channel<TPR, SIDE>(k, i0, 0);
    if (c < D) store_v<8>(p + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (channel<TPR, SIDE>(k, i0, j) < D) p[channel<TPR, SIDE>(k, i0, j)] = from_f32<IT>(v[j]);
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
constexpr int norm_block(int TPR) { return TPR > 32 ? TPR : 256; }
constexpr int norm_rows(int TPR) { return norm_block(TPR) / TPR; }  // rows of a block at a time

// f(parts): the built combination of a call's.
template <typename F>
cudaError_t norm_parts(int parts, F f) {
  constexpr int kGated = kNormPost | kNormGate, kAdd = kNormPre | kNormRes;
  constexpr int kFull = kNormPost | kNormGate | kNormScale | kNormPre | kNormRes;
  if (parts == kGated) return f(std::integral_constant<int, kGated>{});
  if (parts == kAdd) return f(std::integral_constant<int, kAdd>{});
  if (parts == kFull) return f(std::integral_constant<int, kFull>{});
  return f(std::integral_constant<int, kNormAny>{});
}

// f(SIDE): rows of blocks have a kernel of their own for rows that do not take 16-byte accesses (8192 x
// 2047, full backward: 204 us in chunks of 8, 142 us side by side).  The kernel for those that do still asks for
// `vec` at run time: without the question its loads and arithmetic become one block of code, in which
// the compiler orders the next row's loads late (8192 x 4096, full backward: 184 us against 142).
template <int TPR, typename F>
cudaError_t norm_side(int vec, F f) {
  if constexpr (TPR <= 32)
    return f(std::false_type{});
  else
    return vec ? f(std::false_type{}) : f(std::true_type{});
}

gdr_status resolve_norm(const gdr_norm_problem* p, NormDims* d);

struct NormBwdPtrs {
  const void *x, *gate, *r, *dr, *dy;
  const float *w_post, *scale, *w_pre;
  void *dx, *dgate, *dres;
  float* partial;  // [grid][3][D]: dw_post, dscale, dw_pre
};
// The backward's kernel for one pair of types (gdr_norm_bwd_*.cu).  *grid: blocks, lowered to what
// fits the GPU at once.
template <typename IT, typename RT>
cudaError_t norm_bwd_launch(const NormDims& d, const NormBwdPtrs& a, int parts, long long* grid, cudaStream_t s);

}  // namespace gdr
