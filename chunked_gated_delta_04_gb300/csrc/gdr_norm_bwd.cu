// gdr_norm_bwd.cu -- backward of the block norms (include/gdr_block.h):
//
//   with w_pre:   du = dr + rstd(r) (t - rh mean(t rh)),  t = dy w_pre, rh = r rstd(r);  dw_pre = sum dy rh
//   else          du = dr
//   dscale = sum du xh w_post silu(z);   dz = du scale xh w_post silu'(z);
//   t = du scale silu(z);  dw_post = sum t xh;   dx = rstd(x) (t w_post - xh mean(t w_post xh))
//   (dx = t without w_post);  dresidual = du.
//
// One pass: a row stays in registers; its two dependent row sums (the second mean needs du) cost
// two block reductions.  The sums over rows are kept per thread and column for all rows a block
// walks, joined in shared memory where several rows share a block, and written as one partial row
// per block; a second small kernel adds the partial rows in order.
#include "gdr_norm.cuh"

namespace gdr {
namespace {

struct BwdPtrs {
  const void *x, *gate, *r, *dr, *dy;
  const float *w_post, *scale, *w_pre;
  void *dx, *dgate, *dres;
  float* partial;  // [grid][3][D]: dw_post, dscale, dw_pre
};

template <typename IT, typename RT, int TPR, int K>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 256) norm_bwd_kernel(NormDims d, BwdPtrs a) {
  constexpr int kBlock = TPR > 32 ? TPR : 256;
  constexpr int kRowsPerBlock = kBlock / TPR;
  __shared__ float red[TPR > 32 ? 8 * TPR / 32 : 1];  // two buffers of 3 sums, two of 1
  __shared__ float cols[kRowsPerBlock > 1 ? kBlock * 8 : 1];
  int flip = 0, flip1 = 0;
  const int i0 = threadIdx.x % TPR;
  const long long step = (long long)gridDim.x * kRowsPerBlock;
  const float inv = 1.f / (float)d.D;
  float acc[3][K][8];
#pragma unroll
  for (int m = 0; m < 3; ++m)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[m][k][i] = 0.f;
  for (long long base = (long long)blockIdx.x * kRowsPerBlock; base < d.rows; base += step) {
    const long long row = base + threadIdx.x / TPR;
    const long long tok = row / d.heads;
    const int hd = (int)(row - tok * d.heads);
    const int D = row < d.rows ? d.D : 0;  // a dead row loads zeros and stores nothing
    float xv[K][8], du[K][8], rv[K][8], t[8], g[8];
    float s[3] = {0.f, 0.f, 0.f};  // sum x^2, sum r^2, sum dy w_pre r
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = 8 * (k * TPR + i0);
      load8((const IT*)a.x + tok * d.ld_x + (long long)hd * d.D, c, D, d.vec, xv[k]);
      if (a.dr) {
        load8((const RT*)a.dr + row * d.D, c, D, d.vec, du[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) du[k][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] = fmaf(xv[k][i], xv[k][i], s[0]);
      if (a.w_pre) {
        load8((const RT*)a.r + row * d.D, c, D, d.vec, rv[k]);
        load8((const IT*)a.dy + row * d.D, c, D, d.vec, g);
        load8(a.w_pre, c, D, d.vec, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[1] = fmaf(rv[k][i], rv[k][i], s[1]);
          s[2] = fmaf(g[i] * t[i], rv[k][i], s[2]);
        }
      }
    }
    row_sums<TPR, 3>(s, red, flip);
    const float rx = rsqrtf(s[0] * inv + d.eps);
    if (a.w_pre) {
      const float rr = rsqrtf(s[1] * inv + d.eps), m1 = s[2] * inv * rr;  // mean(t rh)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = 8 * (k * TPR + i0);
        load8((const IT*)a.dy + row * d.D, c, D, d.vec, g);  // in the L1 or L2 from above
        load8(a.w_pre, c, D, d.vec, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float rh = rv[k][i] * rr;
          acc[2][k][i] = fmaf(g[i], rh, acc[2][k][i]);
          du[k][i] = fmaf(rr, g[i] * t[i] - rh * m1, du[k][i]);
        }
      }
    }
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = 8 * (k * TPR + i0);
      if (a.dres) store8((RT*)a.dres + row * d.D, c, D, d.vec, du[k]);
      float w[8], z[8], sc[8];
      if (a.w_post) load8(a.w_post, c, D, d.vec, w);
      if (a.scale) load8(a.scale, c, D, d.vec, sc);
      if (a.gate) load8((const IT*)a.gate + tok * d.ld_gate + (long long)hd * d.D, c, D, d.vec, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = a.w_post ? xv[k][i] * rx : xv[k][i];
        const float n = a.w_post ? xh * w[i] : xh;
        float act = 1.f;
        float e = du[k][i];
        if (a.gate) {
          const float sg = sigmoid_f(z[i]);
          act = z[i] * sg;
          t[i] = e * (a.scale ? sc[i] : 1.f) * n * (sg * fmaf(z[i], 1.f - sg, 1.f));
        }
        if (a.scale) {
          acc[1][k][i] = fmaf(e, n * act, acc[1][k][i]);
          e *= sc[i];
        }
        e *= act;
        if (a.w_post) {
          acc[0][k][i] = fmaf(e, xh, acc[0][k][i]);
          e *= w[i];
          q[0] = fmaf(e, xh, q[0]);
        }
        du[k][i] = e;
        xv[k][i] = xh;
      }
      if (a.gate) store8((IT*)a.dgate + row * d.D, c, D, d.vec, t);
    }
    if (a.w_post) {
      row_sums<TPR, 1>(q, red + (TPR > 32 ? 6 * TPR / 32 : 0), flip1);
      const float m2 = q[0] * inv;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) du[k][i] = rx * (du[k][i] - xv[k][i] * m2);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) store8((IT*)a.dx + row * d.D, 8 * (k * TPR + i0), D, d.vec, du[k]);
  }
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    float* out = a.partial + ((long long)blockIdx.x * 3 + m) * d.D;
    if constexpr (kRowsPerBlock == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) store8(out, 8 * (k * TPR + i0), d.D, d.vec, acc[m][k]);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) cols[threadIdx.x * 8 + i] = acc[m][k][i];
        __syncthreads();
        for (int j = threadIdx.x; j < TPR * 8; j += kBlock) {
          float v = 0.f;
#pragma unroll 4
          for (int rw = 0; rw < kRowsPerBlock; ++rw) v += cols[rw * TPR * 8 + j];
          if (8 * k * TPR + j < d.D) out[8 * k * TPR + j] = v;
        }
      }
    }
  }
}

// Blocks of the backward: enough to fill the GPU, few enough that their partial rows stay small
// next to the rows themselves.
long long bwd_grid(const NormDims& d) {
  long long rows_per_block = 1;
  norm_shape(d.D, [&](auto tpr, auto) {
    constexpr int TPR = decltype(tpr)::value;
    rows_per_block = TPR > 32 ? 1 : 256 / TPR;
    return cudaSuccess;
  });
  const long long want = (d.rows + rows_per_block - 1) / rows_per_block, most = 2 * kSmCount;
  return want < most ? want : most;
}

size_t norm_bwd_bytes(const NormDims& d) { return block_align(sizeof(float) * 3 * (size_t)bwd_grid(d) * d.D) + 256; }

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_norm_bwd_workspace_bytes(const gdr_norm_problem* p) {
  NormDims d;
  return resolve_norm(p, &d) == GDR_OK ? norm_bwd_bytes(d) : 0;
}

gdr_status gdr_norm_bwd(const gdr_norm_problem* p, const void* x, const float* w_post, const void* gate,
                        const float* scale, const void* r, const float* w_pre, int has_residual, const void* dr,
                        const void* dy, void* dx, void* dgate, void* dresidual, float* dw_post, float* dscale,
                        float* dw_pre, void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  NormDims d;
  const gdr_status st = resolve_norm(p, &d);
  if (st != GDR_OK) return st;
  if (!w_post && !gate && !scale && !has_residual && !w_pre) return GDR_ERR_INVALID_ARG;
  if (w_pre && !has_residual && (w_post || gate || scale || dr)) return GDR_ERR_INVALID_ARG;
  if (!w_pre != !dy || (!dr && !dy)) return GDR_ERR_INVALID_ARG;
  if (dresidual && !has_residual) return GDR_ERR_INVALID_ARG;
  if ((w_post && !dw_post) || (scale && !dscale) || (w_pre && !dw_pre)) return GDR_ERR_INVALID_ARG;
  if (d.rows > 0 && (!x || !dx || (w_pre && !r) || (gate && !dgate))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype), rel = has_residual ? dtype_bytes(p->res_dtype) : el;
  if (!elem_ok(x, el) || !elem_ok(gate, el) || !elem_ok(dy, el) || !elem_ok(dx, el) || !elem_ok(dgate, el) ||
      !elem_ok(r, rel) || !elem_ok(dr, rel) || !elem_ok(dresidual, rel) || !elem_ok(w_post, 4) || !elem_ok(scale, 4) ||
      !elem_ok(w_pre, 4) || !elem_ok(dw_post, 4) || !elem_ok(dscale, 4) || !elem_ok(dw_pre, 4) ||
      ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < norm_bwd_bytes(d)) return GDR_ERR_WORKSPACE;
  d.vec = d.D % 8 == 0 && d.ld_x % 8 == 0 && d.ld_gate % 8 == 0 && vec_ok(x) && vec_ok(w_post) && vec_ok(gate) &&
          vec_ok(scale) && vec_ok(r) && vec_ok(w_pre) && vec_ok(dr) && vec_ok(dy) && vec_ok(dx) && vec_ok(dgate) &&
          vec_ok(dresidual);
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  float* partial = (float*)workspace;
  const long long grid = bwd_grid(d);
  const BwdPtrs a{x, gate, r, dr, dy, w_post, scale, w_pre, dx, dgate, dresidual, partial};
  auto go = [&](auto it, auto rt) {
    using IT = decltype(it);
    using RT = decltype(rt);
    return norm_shape(d.D, [&](auto tpr, auto k) {
      constexpr int TPR = decltype(tpr)::value, K = decltype(k)::value;
      norm_bwd_kernel<IT, RT, TPR, K><<<(unsigned)grid, TPR > 32 ? TPR : 256, 0, s>>>(d, a);
      stage_mark(s, "norm_bwd");
      return cudaGetLastError();
    });
  };
  if (grid > 0) {
    cudaError_t e;
    if (p->dtype == GDR_DTYPE_F32)
      e = go(float{}, float{});
    else
      e = has_residual && p->res_dtype == GDR_DTYPE_F32 ? go(__nv_bfloat16{}, float{})
                                                         : go(__nv_bfloat16{}, __nv_bfloat16{});
    if (e != cudaSuccess) return status_of(e);
  }
  ColumnSums out = {};
  out.vec[0] = w_post ? dw_post : nullptr;
  out.vec[1] = scale ? dscale : nullptr;
  out.vec[2] = w_pre ? dw_pre : nullptr;
  out.parts = 3;
  out.width = d.D;
  if (!w_post && !scale && !w_pre) return GDR_OK;
  return status_of(launch_column_sums(partial, grid, out, s, "norm_dw"));
}

}  // extern "C"
