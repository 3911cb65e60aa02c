// gdr_attn_simt.cu -- attention in fp32 on the CUDA cores (include/gdr_attn.h): fp32 problems, whose
// accuracy the tensor cores' bf16 and tf32 products do not give, and bf16 ones that are not aligned for TMA.
//
//   forward     per 64 queries of a head, over the visible keys 64 at a time: S = scale Q K^T, running row
//               maximum m and sum l, O <- O e^(m_old - m) + e^(S - m) V;  o = O / l, lse = m + log l
//   backward    P = e^(S - lse), dS = P (dO V^T - delta):
//               per 64 keys of a key head, over its query heads and the queries that see them: dV += P^T dO,
//               dK += scale dS^T Q;  per 64 queries: dQ += scale dS K
// A block is 16 x 16 threads; a thread holds 4 x 4 of S (rows ty + 16 r, columns tx + 16 c) and 4 rows by D / 16
// features of an accumulator.  Bound by the FMA pipes and the shared-memory reads that feed them: 16 products for
// every two 16-byte reads; the next tiles are copied asynchronously beside them.  A third of the pipes' rate is reached: two blocks of eight
// warps an SM, whose barriers and reads are not hidden.  Where there are too few tiles to fill the SMs, the blocks of a cluster share a
// tile: each takes every n-th step of its loop, and each sums the parts of some of the rows from the others' shared memory, in the order
// of their ranks (1903 tokens in four sequences, 4 heads on 2, D = 64: forward 115 -> 46 us, dK and dV 393 -> 77, dQ 143 -> 57, copies
// beside the products and packed sums included).
// T = 4096, causal: fp32, 8 heads of 64, forward 530 us, 32 TFLOP/s, backward 1630 us, 26; of 128, 930 and 3070 us, 37 and 28.  bf16 off 16 bytes,
// 16 heads of 128: 2490 and 7460 us, with loads of single elements, where the tensor cores take 51 and 175 us.
#include "gdr_attn.cuh"
#include "gdr_instrument.cuh"
#include "tc_primitives.cuh"

namespace gdr {
namespace {

constexpr int kT = kSimtTile;
constexpr int kThreads = 256;
constexpr int kPS = kT + 4;  // row stride of a tile of P in floats

// rows [r0, r0 + 64) of a head's [tokens, D] activations to shared memory [64][DP + 4] as fp32, zeros outside; there after
// copy_async_wait and a barrier (copies that pass no registers, where type and alignment allow them).
template <typename IT, int DP>
__device__ __forceinline__ void load_tile(float* dst, const IT* src, long long ld, int r0, int rows, int D) {
  constexpr int S = DP + 4;
  if (sizeof(IT) == 4 && ((uintptr_t)src & 15) == 0 && ld % 4 == 0) {
    for (int e = threadIdx.x; e < kT * (DP / 4); e += kThreads) {
      const int r = e / (DP / 4), c = e % (DP / 4) * 4;
      const bool on = r0 + r < rows && c < D;
      copy_async<16>(dst + r * S + c, on ? src + (long long)(r0 + r) * ld + c : src, on ? 16 : 0);
    }
    return;
  }
  for (int e = threadIdx.x; e < kT * DP; e += kThreads) {
    const int r = e / DP, c = e % DP;
    dst[r * S + c] = r0 + r < rows && c < D ? to_f32(src[(long long)(r0 + r) * ld + c]) : 0.f;
  }
}

// ----------------------------------------------------------------- a cluster's blocks on one tile
__device__ __forceinline__ int cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return (int)n;
}
// A float, or four, at the same place of another block's shared memory.
__device__ __forceinline__ float load_peer(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::mapa(tc::smem_u32(p), (uint32_t)rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_peer4(const float* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(tc::mapa(tc::smem_u32(p), (uint32_t)rank))
               : "memory");
  return v;
}
// Four features of a row (all of them, or none: D is a multiple of 16), times f.
template <typename IT>
__device__ __forceinline__ void store4(IT* p, float4 v, float f) {
  const float x[4] = {v.x * f, v.y * f, v.z * f, v.w * f};
  if ((uintptr_t)p % (4 * sizeof(IT)) == 0) {
    store_v<4>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = from_f32<IT>(x[i]);
  }
}
// Rows 4 ty + r (Column) or ty + 16 r of an accumulator to a tile [64][DP + 4].
template <int DP, bool Column>
__device__ __forceinline__ void put_rows(float* dst, const float (&v)[4][DP / 16], int tx, int ty) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int w = 0; w < DP / 64; ++w)
      *reinterpret_cast<float4*>(dst + (Column ? 4 * ty + r : ty + 16 * r) * (DP + 4) + 4 * tx + 64 * w) =
          make_float4(v[r][4 * w], v[r][4 * w + 1], v[r][4 * w + 2], v[r][4 * w + 3]);
}
// Rows of this block's share of a tile, summed over the cluster's blocks, times f to `out` (row `first` on at out, D features).
template <typename IT, int DP>
__device__ __forceinline__ void sum_rows(const float* tile, int rank, int n, IT* out, long long ld, int rows, int D, float f) {
  const int r0 = kT * rank / n, r1 = min(rows, kT * (rank + 1) / n);
  for (int e = threadIdx.x; e < (r1 - r0) * (DP / 4); e += kThreads) {
    const int r = r0 + e / (DP / 4), c = e % (DP / 4) * 4;
    if (c >= D) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < n; ++x) {
      const float4 v = load_peer4(tile + r * (DP + 4) + c, x);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    store4(out + (long long)r * ld + c, sum, f);
  }
}

// acc[r][c] = A[ty + 16 r] . B[tx + 16 c] over the DP features; even and odd ones in the halves of a packed sum, which takes half the
// instructions.
template <int DP>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int tx, int ty, float (&acc)[4][4]) {
  constexpr int S = DP + 4;
  f32x2 sum[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[r][c] = 0;  // a pair of zeros
#pragma unroll 4
  for (int k = 0; k < DP; k += 4) {
    ulonglong2 a[4], b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const ulonglong2*>(A + (ty + 16 * r) * S + k);
#pragma unroll
    for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * c) * S + k);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[r][c] = fma2(a[r].y, b[c].y, fma2(a[r].x, b[c].x, sum[r][c]));
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[r][c] = lo2(sum[r][c]) + hi2(sum[r][c]);
}

// out[r][.] += sum_j M[ty + 16 r][j] X[j][features 4 tx + 64 w ..]: M [64][kPS], X [64][DP + 4].
template <int DP>
__device__ __forceinline__ void row_product(const float* M, const float* X, int tx, int ty, float (&out)[4][DP / 16]) {
  constexpr int S = DP + 4;
#pragma unroll 2
  for (int j = 0; j < kT; j += 4) {
    float4 p[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4*>(M + (ty + 16 * r) * kPS + j);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int w = 0; w < DP / 64; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(X + (j + jj) * S + 4 * tx + 64 * w);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float pr = jj == 0 ? p[r].x : jj == 1 ? p[r].y : jj == 2 ? p[r].z : p[r].w;
          out[r][4 * w] = fmaf(pr, x.x, out[r][4 * w]);
          out[r][4 * w + 1] = fmaf(pr, x.y, out[r][4 * w + 1]);
          out[r][4 * w + 2] = fmaf(pr, x.z, out[r][4 * w + 2]);
          out[r][4 * w + 3] = fmaf(pr, x.w, out[r][4 * w + 3]);
        }
      }
  }
}

// out[r][.] += sum_i M[i][4 ty + r] X[i][features 4 tx + 64 w ..].
template <int DP>
__device__ __forceinline__ void column_product(const float* M, const float* X, int tx, int ty, float (&out)[4][DP / 16]) {
  constexpr int S = DP + 4;
#pragma unroll 4
  for (int i = 0; i < kT; ++i) {
    const float4 p = *reinterpret_cast<const float4*>(M + i * kPS + 4 * ty);
#pragma unroll
    for (int w = 0; w < DP / 64; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(X + i * S + 4 * tx + 64 * w);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float pr = r == 0 ? p.x : r == 1 ? p.y : r == 2 ? p.z : p.w;
        out[r][4 * w] = fmaf(pr, x.x, out[r][4 * w]);
        out[r][4 * w + 1] = fmaf(pr, x.y, out[r][4 * w + 1]);
        out[r][4 * w + 2] = fmaf(pr, x.z, out[r][4 * w + 2]);
        out[r][4 * w + 3] = fmaf(pr, x.w, out[r][4 * w + 3]);
      }
    }
  }
}

// An accumulator's row: features 4 tx + 64 w .. of it, times f.
template <typename IT, int DP>
__device__ __forceinline__ void store_row(IT* dst, const float (&v)[DP / 16], float f, int tx, int D) {
#pragma unroll
  for (int w = 0; w < DP / 64; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = 4 * tx + 64 * w + e;
      if (c < D) dst[c] = from_f32<IT>(v[4 * w + e] * f);
    }
}

template <int DP>
constexpr size_t tile_bytes() { return sizeof(float) * kT * (DP + 4); }

// Whether some query of a tile does not see some key of it.
__device__ __forceinline__ bool partial(const AttnDims& d, const AttnSpan& s, int off, int i0, int j0) {
  return j0 + kT > s.m || (d.causal && j0 + kT - 1 > i0 + off) || (d.window && j0 <= i0 + kT - 1 + off - d.window);
}

template <typename IT, int DP>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1) attn_fwd_simt_kernel(AttnDims d, AttnTiles t, AttnFwdArgs a) {
  extern __shared__ float smem[];
  float *Q = smem, *K = Q + kT * (DP + 4), *V = K + kT * (DP + 4), *P = V + kT * (DP + 4);
  launch_wait();
  launch_next();
  if (blockIdx.x == 0 && threadIdx.x == 0 && !d.cu_q) *a.status = 0;  // of a packed batch: the tile table's kernel
  int seq, h, tile;
  const int n = cluster_size(), rank = n > 1 ? (int)tc::cluster_ctarank() : 0;
  if (!attn_tile(d, t, d.Hq, blockIdx.x / n, &seq, &h, &tile)) return;
  const AttnSpan s = attn_span(d, seq);
  const int i0 = tile * kT, off = s.m - s.n, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (i0 >= s.n) return;
  const IT* q = (const IT*)a.q + s.q0 * d.ld_q + (long long)h * d.D;
  const IT* k = (const IT*)a.k + s.k0 * d.ld_k + (long long)(h / d.G) * d.D;
  const IT* v = (const IT*)a.v + s.k0 * d.ld_v + (long long)(h / d.G) * d.D;
  load_tile<IT, DP>(Q, q, d.ld_q, i0, s.n, d.D);
  float O[4][DP / 16] = {}, m[4], l[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = 0.f;
  int lo, hi;
  attn_keys(d, s, i0, min(s.n, i0 + kT), &lo, &hi);
  const float c = d.scale * kLog2e;
  const int begin = (lo / kT + rank) * kT;
  if (begin < hi) load_tile<IT, DP>(K, k, d.ld_k, begin, s.m, d.D);
  for (int j0 = begin; j0 < hi; j0 += kT * n) {
    copy_async_wait();
    __syncthreads();  // the keys are here, and the values and P of the step before used up
    GDR_DELAY_WARP(63);
    load_tile<IT, DP>(V, v, d.ld_v, j0, s.m, d.D);
    float S[4][4];
    dot_tile<DP>(Q, K, tx, ty, S);
    if (partial(d, s, off, i0, j0))
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + tx + 16 * e;
          if (j >= s.m || !attn_sees(d, off, i0 + ty + 16 * r, j)) S[r][e] = -INFINITY;
        }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // (a NaN passes the maximum by and reaches the row through its own exponential)
      float top = fmaxf(fmaxf(fmaxf(m[r], S[r][0]), fmaxf(S[r][1], S[r][2])), S[r][3]);
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = attn_base(top, c), f = attn_rescale(m[r], c, base);
      m[r] = top;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = ex2f(fmaf(S[r][e], c, -base));
        sum += p;
        P[(ty + 16 * r) * kPS + tx + 16 * e] = p;
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[r] = fmaf(l[r], f, sum);
#pragma unroll
      for (int e = 0; e < DP / 16; ++e) O[r][e] *= f;
    }
    copy_async_wait();
    __syncthreads();
    if (j0 + kT * n < hi) load_tile<IT, DP>(K, k, d.ld_k, j0 + kT * n, s.m, d.D);
    row_product<DP>(P, V, tx, ty, O);
  }
  if (n > 1) {  // every block's O, maxima and sums; then the rows of its share from all of them
    __syncthreads();
    put_rows<DP, false>(K, O, tx, ty);
    if (tx == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) P[ty + 16 * r] = m[r], P[kT + ty + 16 * r] = l[r];
    GDR_DELAY_WARP(64);
    tc::cluster_sync();
    const int r0 = kT * rank / n, r1 = kT * (rank + 1) / n;
    for (int e = threadIdx.x; e < (r1 - r0) * (DP / 4); e += kThreads) {
      const int r = r0 + e / (DP / 4), x = e % (DP / 4) * 4, i = i0 + r;
      if (i >= s.n || x >= d.D) continue;
      float top = -INFINITY, sum = 0.f;
      for (int y = 0; y < n; ++y) top = fmaxf(top, load_peer(P + r, y));
      const float base = attn_base(top, c);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int y = 0; y < n; ++y) {
        const float f = attn_rescale(load_peer(P + r, y), c, base);
        const float4 v = load_peer4(K + r * (DP + 4) + x, y);
        sum = fmaf(load_peer(P + kT + r, y), f, sum);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
      }
      const bool none = top == -INFINITY && sum == 0.f;
      store4((IT*)a.o + (s.q0 + i) * (long long)d.Hq * d.D + (long long)h * d.D + x, none ? make_float4(0.f, 0.f, 0.f, 0.f) : o,
             none ? 0.f : 1.f / sum);
      if (x == 0) a.lse[s.lse0 + (long long)h * d.Tq + i] = none ? -INFINITY : fmaf(top, d.scale, logf(sum));
    }
    tc::cluster_sync();  // no block ends while others read it
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + ty + 16 * r;
    if (i >= s.n) continue;
    store_row<IT, DP>((IT*)a.o + (s.q0 + i) * (long long)d.Hq * d.D + (long long)h * d.D, O[r], m[r] == -INFINITY && l[r] == 0.f ? 0.f : 1.f / l[r], tx, d.D);
    if (tx == 0)
      a.lse[s.lse0 + (long long)h * d.Tq + i] = m[r] == -INFINITY && l[r] == 0.f ? -INFINITY : fmaf(m[r], d.scale, logf(l[r]));
  }
}

// P and dS of a tile: rows i0 .., columns j0 .. of a sequence.
template <int DP>
__device__ __forceinline__ void grad_tile(const AttnDims& d, const AttnSpan& s, int i0, int j0, const float* Q, const float* K,
                                          const float* dO, const float* V, const float* lse, const float* delta, int tx, int ty,
                                          float (&p)[4][4], float (&ds)[4][4]) {
  const int off = s.m - s.n;
  dot_tile<DP>(Q, K, tx, ty, p);
  dot_tile<DP>(dO, V, tx, ty, ds);
  const bool cut = i0 + kT > s.n || partial(d, s, off, i0, j0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + ty + 16 * r;
    const float ls = i < s.n ? lse[i] : 0.f, dl = i < s.n ? delta[i] : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[r][e] = ex2f(kLog2e * fmaf(p[r][e], d.scale, -ls));
      ds[r][e] = p[r][e] * (ds[r][e] - dl);
    }
    if (cut)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + tx + 16 * e;
        if (i >= s.n || j >= s.m || !attn_sees(d, off, i, j)) p[r][e] = ds[r][e] = 0.f;
      }
  }
}

__device__ __forceinline__ void put_tile(float* dst, const float (&v)[4][4], int tx, int ty) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) dst[(ty + 16 * r) * kPS + tx + 16 * e] = v[r][e];
}

template <typename IT, int DP>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1) attn_dkdv_simt_kernel(AttnDims d, AttnTiles t, AttnBwdArgs a) {
  extern __shared__ float smem[];
  constexpr int N = kT * (DP + 4);
  float *K = smem, *V = K + N, *Q = V + N, *dO = Q + N, *Qn = dO + N, *M = Qn + N;  // Qn: the next step's
  launch_wait();
  launch_next();
  int seq, h, tile;
  const int n = cluster_size(), rank = n > 1 ? (int)tc::cluster_ctarank() : 0;
  if (!attn_tile(d, t, d.Hk, blockIdx.x / n, &seq, &h, &tile)) return;
  const AttnSpan s = attn_span(d, seq);
  const int j0 = tile * kT, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (j0 >= s.m) return;
  load_tile<IT, DP>(K, (const IT*)a.k + s.k0 * d.ld_k + (long long)h * d.D, d.ld_k, j0, s.m, d.D);
  load_tile<IT, DP>(V, (const IT*)a.v + s.k0 * d.ld_v + (long long)h * d.D, d.ld_v, j0, s.m, d.D);
  float dK[4][DP / 16] = {}, dV[4][DP / 16] = {};
  int lo, hi;
  attn_queries(d, s, j0, min(s.m, j0 + kT), &lo, &hi);
  const int first = lo / kT, length = lo < hi ? (hi + kT - 1) / kT - first : 0, steps = length * d.G;
  // queries and gradients of a step: query head and first query
  auto at_step = [&](int st, int* hq, int* i0) {
    *hq = h * d.G + st / length;
    *i0 = (first + st % length) * kT;
  };
  auto load = [&](float* dst, const void* from, long long ld, int st) {
    int hq, i0;
    at_step(st, &hq, &i0);
    load_tile<IT, DP>(dst, (const IT*)from + s.q0 * ld + (long long)hq * d.D, ld, i0, s.n, d.D);
  };
  if (rank < steps) {
    load(Q, a.q, d.ld_q, rank);
    load(dO, a.dout, d.ld_do, rank);
  }
  for (int st = rank; st < steps; st += n) {
    int hq, i0;
    at_step(st, &hq, &i0);
    const long long stat = s.lse0 + (long long)hq * d.Tq;
    copy_async_wait();
    __syncthreads();
    GDR_DELAY_WARP(63);
    if (st + n < steps) load(Qn, a.q, d.ld_q, st + n);
    float p[4][4], ds[4][4];
    grad_tile<DP>(d, s, i0, j0, Q, K, dO, V, a.lse + stat, a.delta + stat, tx, ty, p, ds);
    put_tile(M, p, tx, ty);
    __syncthreads();
    column_product<DP>(M, dO, tx, ty, dV);
    __syncthreads();
    if (st + n < steps) load(dO, a.dout, d.ld_do, st + n);
    put_tile(M, ds, tx, ty);
    __syncthreads();
    column_product<DP>(M, Q, tx, ty, dK);
    float* const t = Q;
    Q = Qn;
    Qn = t;
  }
  if (n > 1) {
    __syncthreads();
    Q = smem + 2 * N;  // the same place in every block, whichever it had last
    put_rows<DP, true>(Q, dK, tx, ty);
    put_rows<DP, true>(dO, dV, tx, ty);
    GDR_DELAY_WARP(64);
    tc::cluster_sync();
    const long long at = (s.k0 + j0) * (long long)d.Hk * d.D + (long long)h * d.D, ld = (long long)d.Hk * d.D;
    sum_rows<IT, DP>(Q, rank, n, (IT*)a.dk + at, ld, s.m - j0, d.D, d.scale);
    sum_rows<IT, DP>(dO, rank, n, (IT*)a.dv + at, ld, s.m - j0, d.D, 1.f);
    tc::cluster_sync();  // no block ends while others read it
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = j0 + 4 * ty + r;
    if (j >= s.m) continue;
    const long long at = (s.k0 + j) * (long long)d.Hk * d.D + (long long)h * d.D;
    store_row<IT, DP>((IT*)a.dk + at, dK[r], d.scale, tx, d.D);
    store_row<IT, DP>((IT*)a.dv + at, dV[r], 1.f, tx, d.D);
  }
}

template <typename IT, int DP>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1) attn_dq_simt_kernel(AttnDims d, AttnTiles t, AttnBwdArgs a) {
  extern __shared__ float smem[];
  constexpr int N = kT * (DP + 4);
  float *Q = smem, *dO = Q + N, *K = dO + N, *V = K + N, *Kn = V + N, *M = Kn + N;  // Kn: the next step's
  launch_wait();
  launch_next();
  int seq, h, tile;
  const int n = cluster_size(), rank = n > 1 ? (int)tc::cluster_ctarank() : 0;
  if (!attn_tile(d, t, d.Hq, blockIdx.x / n, &seq, &h, &tile)) return;
  const AttnSpan s = attn_span(d, seq);
  const int i0 = tile * kT, hk = h / d.G, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (i0 >= s.n) return;
  const long long stat = s.lse0 + (long long)h * d.Tq;
  load_tile<IT, DP>(Q, (const IT*)a.q + s.q0 * d.ld_q + (long long)h * d.D, d.ld_q, i0, s.n, d.D);
  load_tile<IT, DP>(dO, (const IT*)a.dout + s.q0 * d.ld_do + (long long)h * d.D, d.ld_do, i0, s.n, d.D);
  float dQ[4][DP / 16] = {};
  int lo, hi;
  attn_keys(d, s, i0, min(s.n, i0 + kT), &lo, &hi);
  const IT* const k = (const IT*)a.k + s.k0 * d.ld_k + (long long)hk * d.D;
  const IT* const v = (const IT*)a.v + s.k0 * d.ld_v + (long long)hk * d.D;
  const int begin = (lo / kT + rank) * kT;
  if (begin < hi) {
    load_tile<IT, DP>(K, k, d.ld_k, begin, s.m, d.D);
    load_tile<IT, DP>(V, v, d.ld_v, begin, s.m, d.D);
  }
  for (int j0 = begin; j0 < hi; j0 += kT * n) {
    const bool more = j0 + kT * n < hi;
    copy_async_wait();
    __syncthreads();
    GDR_DELAY_WARP(63);
    if (more) load_tile<IT, DP>(Kn, k, d.ld_k, j0 + kT * n, s.m, d.D);
    float p[4][4], ds[4][4];
    grad_tile<DP>(d, s, i0, j0, Q, K, dO, V, a.lse + stat, a.delta + stat, tx, ty, p, ds);
    put_tile(M, ds, tx, ty);
    __syncthreads();
    if (more) load_tile<IT, DP>(V, v, d.ld_v, j0 + kT * n, s.m, d.D);
    row_product<DP>(M, K, tx, ty, dQ);
    float* const t = K;
    K = Kn;
    Kn = t;
  }
  if (n > 1) {
    __syncthreads();
    K = smem + 2 * N;  // the same place in every block, whichever it had last
    put_rows<DP, false>(K, dQ, tx, ty);
    GDR_DELAY_WARP(64);
    tc::cluster_sync();
    const long long at = (s.q0 + i0) * (long long)d.Hq * d.D + (long long)h * d.D;
    sum_rows<IT, DP>(K, rank, n, (IT*)a.dq + at, (long long)d.Hq * d.D, s.n - i0, d.D, d.scale);
    tc::cluster_sync();  // no block ends while others read it
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + ty + 16 * r;
    if (i < s.n) store_row<IT, DP>((IT*)a.dq + (s.q0 + i) * (long long)d.Hq * d.D + (long long)h * d.D, dQ[r], d.scale, tx, d.D);
  }
}

// resident: blocks that an SM holds; steps: of the longest tile's loop.  Blocks of a cluster: as many as it takes to give every SM its
// blocks, at most 8, and no more than there are steps.
template <typename F, typename A>
cudaError_t go(F kernel, long long items, size_t smem, int resident, long long steps, const AttnDims& d, const AttnTiles& t, const A& a,
               cudaStream_t s, const char* stage) {
  if (items == 0) return cudaSuccess;
  cudaError_t e = set_smem_once((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  int n = 1;
  while (n < 8 && items * n < (long long)resident * kSmCount && 2 * n <= steps) n *= 2;
  e = attn_launch(kernel, items * n, kThreads, smem, n, s, d, t, a);
  if (e != cudaSuccess) return e;
  stage_mark(s, stage);
  return cudaGetLastError();
}

template <typename IT, int DP>
cudaError_t fwd(const AttnDims& d, const AttnTiles& t, const AttnFwdArgs& a, cudaStream_t s) {
  return go(attn_fwd_simt_kernel<IT, DP>, attn_tile_count(d, false, kT) * d.Hq, 3 * tile_bytes<DP>() + sizeof(float) * kT * kPS, DP == 64 ? 2 : 1,
            (d.Tk + kT - 1) / kT, d, t, a, s, "attn_fwd");
}
template <typename IT, int DP>
cudaError_t bwd(const AttnDims& d, const AttnTiles& tq, const AttnTiles& tk, const AttnBwdArgs& a, cudaStream_t s) {
  constexpr size_t smem = 5 * tile_bytes<DP>() + sizeof(float) * kT * kPS;
  constexpr int resident = DP == 64 ? 2 : 1;
  const cudaError_t e = go(attn_dkdv_simt_kernel<IT, DP>, attn_tile_count(d, true, kT) * d.Hk, smem, resident,
                           (long long)((d.Tq + kT - 1) / kT) * d.G, d, tk, a, s, "attn_dkdv");
  if (e != cudaSuccess) return e;
  return go(attn_dq_simt_kernel<IT, DP>, attn_tile_count(d, false, kT) * d.Hq, smem, resident, (d.Tk + kT - 1) / kT, d, tq, a, s, "attn_dq");
}

}  // namespace

cudaError_t launch_attn_fwd_simt(const AttnDims& d, const AttnTiles& t, bool bf16, const AttnFwdArgs& a, cudaStream_t s) {
  if (bf16) return d.D > 64 ? fwd<__nv_bfloat16, 128>(d, t, a, s) : fwd<__nv_bfloat16, 64>(d, t, a, s);
  return d.D > 64 ? fwd<float, 128>(d, t, a, s) : fwd<float, 64>(d, t, a, s);
}

cudaError_t launch_attn_bwd_simt(const AttnDims& d, const AttnTiles& tq, const AttnTiles& tk, bool bf16, const AttnBwdArgs& a,
                                 cudaStream_t s) {
  if (bf16) return d.D > 64 ? bwd<__nv_bfloat16, 128>(d, tq, tk, a, s) : bwd<__nv_bfloat16, 64>(d, tq, tk, a, s);
  return d.D > 64 ? bwd<float, 128>(d, tq, tk, a, s) : bwd<float, 64>(d, tq, tk, a, s);
}

}  // namespace gdr
