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

// Blocks of the backward: enough to fill the GPU, few enough that their partial rows stay small
// next to the rows themselves.
long long bwd_grid(const NormDims& d) {
  long long rows = 1, per_sm = 1;
  norm_shape(d.D, [&](auto tpr, auto) {
    rows = norm_rows(decltype(tpr)::value);
    per_sm = 1024 / norm_block(decltype(tpr)::value);
    return cudaSuccess;
  });
  const long long want = (d.rows + rows - 1) / rows, most = per_sm * kSmCount;
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
  if ((w_post && !dw_post) || (scale && !dscale) || (w_pre && !dw_pre)) return GDR_ERR_INVALID_ARG;
  if (d.rows > 0) {  // tensors of no rows may have no address
    if (!w_post && !gate && !scale && !has_residual && !w_pre) return GDR_ERR_INVALID_ARG;
    if (w_pre && !has_residual && (w_post || gate || scale || dr)) return GDR_ERR_INVALID_ARG;
    if (!w_pre != !dy || (!dr && !dy)) return GDR_ERR_INVALID_ARG;
    if (dresidual && !has_residual) return GDR_ERR_INVALID_ARG;
    if (!x || !dx || (w_pre && !r) || (gate && !dgate)) return GDR_ERR_INVALID_ARG;
  }
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
  long long grid = bwd_grid(d);
  const NormBwdPtrs a{x, gate, r, dr, dy, w_post, scale, w_pre, dx, dgate, dresidual, partial};
  if (grid > 0) {
    const int parts = (w_post ? kNormPost : 0) | (gate ? kNormGate : 0) | (scale ? kNormScale : 0) |
                      (w_pre ? kNormPre : 0) | (has_residual ? kNormRes : 0);
    cudaError_t e;
    if (p->dtype == GDR_DTYPE_F32)
      e = norm_bwd_launch<float, float>(d, a, parts, &grid, s);
    else if (has_residual && p->res_dtype == GDR_DTYPE_F32)
      e = norm_bwd_launch<__nv_bfloat16, float>(d, a, parts, &grid, s);
    else
      e = norm_bwd_launch<__nv_bfloat16, __nv_bfloat16>(d, a, parts, &grid, s);
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
