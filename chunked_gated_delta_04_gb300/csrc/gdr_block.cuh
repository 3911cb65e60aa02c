// gdr_block.cuh -- what the operators of include/gdr_block.h share: vector access, activations,
// the sequence check of packed batches, the column reduction of parameter gradients.
#pragma once

#include "../../include/gdr_block.h"
#include "gdr_device.cuh"
#include "gdr_internal.h"

namespace gdr {

constexpr int kSmCount = 152;  // SMs of a GB300: grids are sized against it

// Stores of V elements of one row from fp32: vector accesses for V = 4 and 8, scalar for V = 1.  p is aligned to
// the access (at most 16 bytes).
template <int V>
__device__ __forceinline__ void store_v(float* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    p[0] = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    p[0] = __float2bfloat16_rn(v[0]);
  } else if constexpr (V == 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x).  e^-x overflows to infinity below -88, where the reciprocal gives 0, the limit.
__device__ __forceinline__ float sigmoid_f(float x) { return rcpf(1.f + ex2f(-kLog2e * x)); }

// softplus(x) = max(x, 0) + log(1 + u), u = e^-|x| in (0, 1], to fp32 accuracy also where it is
// tiny: log(1 + u) = 2 artanh(s), s = u / (2 + u) <= 1/3, and artanh(s) / s is within 1e-8 of this
// polynomial in s^2 on [0, 1/9] (least maximal relative error, fitted in 64 bits, then rounded).
__host__ __device__ constexpr float artanh_c(int i) {
  return i == 0 ? 1.f : i == 1 ? 0.33333155512809753f : i == 2 ? 0.20012478530406952f : i == 3 ? 0.13979974389076233f
                                                                                       : 0.1409064382314682f;
}
// *sig (nullable) receives sigmoid(x).
__device__ __forceinline__ float softplus_f(float x, float* sig) {
  const float u = ex2f(-kLog2e * fabsf(x));
  const float s = u * rcpf(2.f + u), q = s * s;
  float p = artanh_c(4);
#pragma unroll
  for (int i = 3; i >= 0; --i) p = fmaf(p, q, artanh_c(i));
  if (sig) {
    const float r = rcpf(1.f + u);
    *sig = x >= 0.f ? r : u * r;
  }
  return fmaf(2.f * s, p, fmaxf(x, 0.f));
}

// Two fp32 values in a register pair, for the packed fp32 instructions.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lo2(f32x2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(f32x2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) { return pack2(ex2f(lo2(v)), ex2f(hi2(v))); }

// Sigmoids of a pair.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 v) {
  const f32x2 d = add2(ex2_2(mul2(v, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f));
  return pack2(rcpf(lo2(d)), rcpf(hi2(d)));
}

// The sequence of packed token t (cu valid, t < cu[num_seqs]): the last n with cu[n] <= t.
__device__ __forceinline__ int seq_of(const int32_t* cu, int num_seqs, long long t) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// Copies `bytes` (4, 8 or 16; the rest of a Bytes-wide destination is zeros) without passing registers.
template <int Bytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src), "n"(Bytes), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `Left` of the groups committed last are under way.
template <int Left>
__device__ __forceinline__ void copy_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(Left) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

inline size_t block_align(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool vec_ok(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool elem_ok(const void* p, size_t el) { return ((uintptr_t)p & (el - 1)) == 0; }
inline bool dtype_ok(gdr_dtype t) { return t == GDR_DTYPE_F32 || t == GDR_DTYPE_BF16; }
inline size_t dtype_bytes(gdr_dtype t) { return t == GDR_DTYPE_BF16 ? 2 : 4; }

// Blocks of a kernel that fit on an SM together (asked once per kernel).
template <typename F>
inline int resident_blocks(F kernel, int threads, size_t smem = 0) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();  // our own query's error
    n = 1;
  }
  return n;
}

// Checks cu_seqlens (0 .. T, non-decreasing) and writes status word 0: 0, or the bad bit, on which
// the kernels that follow return at once.
cudaError_t launch_seq_check(const int32_t* cu, int num_seqs, int T, uint32_t* status, cudaStream_t s);

// Sums over the rows of partial[rows][parts][width], in a fixed order: parts k < mat_parts go to
// mat[c * mat_parts + k], the others to vec[k - mat_parts][c] (skipped where null).
struct ColumnSums {
  float* mat;
  int mat_parts;
  float* vec[3];
  int parts, width;
  const uint32_t* status;  // nullable: nothing is written where the sequence check's word is set
};
cudaError_t launch_column_sums(const float* partial, long long rows, const ColumnSums& out, cudaStream_t s,
                               const char* stage);

}  // namespace gdr
