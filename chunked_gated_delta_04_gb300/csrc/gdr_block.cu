// gdr_block.cu -- kernels that several operators of include/gdr_block.h use.
#include "gdr_block.cuh"

namespace gdr {
namespace {

__global__ void __launch_bounds__(256) seq_check_kernel(const int32_t* __restrict__ cu, int num_seqs, int T,
                                                        uint32_t* __restrict__ status) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = cu[0] != 0 || cu[num_seqs] != T;
  __syncthreads();
  for (int n = threadIdx.x; n < num_seqs; n += blockDim.x)
    if (cu[n] > cu[n + 1]) bad = 1;
  __syncthreads();
  if (threadIdx.x == 0) status[0] = bad ? kDevErrBadCuSeqlens : 0u;
}

// 32 columns x G row groups per block; a thread sums every G-th row in order, then the sums are
// added in order: the same result on every run.  G = 32 where there are rows enough (456 rows of
// 384 columns: 4 us against 10 us with 8), 8 where there are few (32 rows of 30720: 9 us against 21 with 32).
template <int G>
__global__ void __launch_bounds__(32 * G) column_sums_kernel(const float* __restrict__ partial, long long rows,
                                                           ColumnSums out) {
  __shared__ float part[G][33];
  if (out.status && *out.status) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long long cols = (long long)out.parts * out.width, col = (long long)blockIdx.x * 32 + x;
  const int k = (int)(col / out.width), c = (int)(col - (long long)k * out.width);
  float* to = col >= cols ? nullptr : k < out.mat_parts ? out.mat + (long long)c * out.mat_parts + k
                                    : out.vec[k - out.mat_parts] ? out.vec[k - out.mat_parts] + c : nullptr;
  float a = 0.f;
  if (to) {
    long long r = y;
    for (; r + 3 * G < rows; r += 4 * G) {
      const float v0 = partial[r * cols + col], v1 = partial[(r + G) * cols + col];
      const float v2 = partial[(r + 2 * G) * cols + col], v3 = partial[(r + 3 * G) * cols + col];
      a += v0;
      a += v1;
      a += v2;
      a += v3;
    }
    for (; r < rows; r += G) a += partial[r * cols + col];
  }
  part[y][x] = a;
  __syncthreads();
  if (y == 0 && to) {
#pragma unroll
    for (int i = 1; i < G; ++i) a += part[i][x];
    *to = a;
  }
}

}  // namespace

cudaError_t launch_seq_check(const int32_t* cu, int num_seqs, int T, uint32_t* status, cudaStream_t s) {
  seq_check_kernel<<<1, 256, 0, s>>>(cu, num_seqs, T, status);
  stage_mark(s, "seq_check");
  return cudaGetLastError();
}

cudaError_t launch_column_sums(const float* partial, long long rows, const ColumnSums& out, cudaStream_t s,
                               const char* stage) {
  const long long cols = (long long)out.parts * out.width;
  if (cols == 0) return cudaSuccess;
  const unsigned grid = (unsigned)((cols + 31) / 32);
  if (rows >= 128)
    column_sums_kernel<32><<<grid, 1024, 0, s>>>(partial, rows, out);
  else
    column_sums_kernel<8><<<grid, 256, 0, s>>>(partial, rows, out);
  stage_mark(s, stage);
  return cudaGetLastError();
}

}  // namespace gdr
