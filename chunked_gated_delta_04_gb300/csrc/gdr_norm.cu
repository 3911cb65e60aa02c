// gdr_norm.cu -- norms before and after a block with its gate and residual scale, forward
// (include/gdr_block.h):
//
//   u = x [rstd(x) w_post] [silu(z)] [scale],   r = [residual +] u,   y = r rstd(r) w_pre
//
// in one pass: a row stays in registers from its load to the store of r and y, so the bytes are
// those of the tensors once each.  Bound by memory (about 10 operations per element): residual add and
// norm of 8192 x 2048 bf16 22.5 us, 6.0 TB/s; gated norm of 131072 x 128 20.6 us, 4.9 TB/s.  The norm
// before the block is taken of r as stored (rounded to its type): the backward, which gets r and
// not the unrounded sum, then differentiates exactly what ran.
#include "gdr_norm.cuh"

namespace gdr {
namespace {

struct FwdPtrs {
  const void *x, *gate, *residual;
  const float *w_post, *scale, *w_pre;
  void *r, *y;
};

// Blocks per SM to fit the registers to (0: the compiler's choice).  Rows of 512 threads with everything
// take 72 registers unasked, which leaves one block per SM: 8192 x 4096, bf16 with an fp32 stream, 108 us; with 64
// registers and two blocks 80 us.  In fp32, where the cap was not measured against none, it costs 44 to 56
// bytes of spills in the general kernel and with everything.  Wider rows spill without a cap (above 8192 channels 36 to
// 280 bytes in bf16, up to 3.7 KB in fp32: 2048 x 16384, everything, fp32 267 us, where the bytes are 100); narrower ones
// are better off unasked (8192 x 2048, add: 22.4 us against 23.6).
constexpr int fwd_min_blocks(int TPR, int K) { return TPR == 512 && K == 1 ? 2 : 0; }

// A block walks rows and has the next ones' loads in flight while it works on the present ones.
template <typename IT, typename RT, int TPR, int K, int PARTS, bool SIDE>
__global__ void __launch_bounds__(norm_block(TPR), fwd_min_blocks(TPR, K)) norm_fwd_kernel(NormDims d, FwdPtrs a) {
  constexpr int kRows = norm_rows(TPR);
  __shared__ float red[TPR > 32 ? 2 * TPR / 32 : 1];
  int flip = 0;
  const bool post = PARTS >= 0 ? (PARTS & kNormPost) != 0 : a.w_post != nullptr;
  const bool gate = PARTS >= 0 ? (PARTS & kNormGate) != 0 : a.gate != nullptr;
  const bool scale = PARTS >= 0 ? (PARTS & kNormScale) != 0 : a.scale != nullptr;
  const bool pre = PARTS >= 0 ? (PARTS & kNormPre) != 0 : a.w_pre != nullptr;
  const bool res = PARTS >= 0 ? (PARTS & kNormRes) != 0 : a.residual != nullptr;
  const int i0 = threadIdx.x % TPR;
  const float inv = 1.f / (float)d.D;
  struct Row {
    Raw8<IT> x[K], z[K];
    Raw8<RT> res[K];
  };
  auto load = [&](long long row, Row& o) {
    const int D = row < d.rows ? d.D : 0;  // a missing row is zeros and is not stored
    const long long tok = token_of(d, row), at = (row - tok * d.heads) * d.D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      o.x[k] = load_raw8<TPR, SIDE>((const IT*)a.x + tok * d.ld_x + at, k, i0, D, d.vec);
      if (gate) o.z[k] = load_raw8<TPR, SIDE>((const IT*)a.gate + tok * d.ld_gate + at, k, i0, D, d.vec);
      if (res) o.res[k] = load_raw8<TPR, SIDE>((const RT*)a.residual + row * d.D, k, i0, D, d.vec);
    }
  };
  // rows of a block run together (barriers): the loop's trip count is the block's
  const long long step = (long long)gridDim.x * kRows;
  long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  Row cur;
  load(row, cur);
  for (long long base = (long long)blockIdx.x * kRows; base < d.rows; base += step, row += step) {
    Row next;
    if (base + step < d.rows) load(row + step, next);
    const int D = row < d.rows ? d.D : 0;
    float u[K][8], t[8];
#pragma unroll
    for (int k = 0; k < K; ++k) cur.x[k].get(u[k]);
    if (post) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(u[k][i], u[k][i], s[0]);
      row_sums<TPR, 1>(s, red, flip);
      const float rs = rsqrtf(s[0] * inv + d.eps);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        load_raw8<TPR, SIDE>(a.w_post, k, i0, D, d.vec).get(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] *= rs * t[i];
      }
    }
    if (gate) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        cur.z[k].get(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] *= t[i] * sigmoid_f(t[i]);
      }
    }
    if (scale) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        load_raw8<TPR, SIDE>(a.scale, k, i0, D, d.vec).get(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] *= t[i];
      }
    }
    if (res) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        cur.res[k].get(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] = to_f32(from_f32<RT>(u[k][i] + t[i]));
        store8<TPR, SIDE>((RT*)a.r + row * d.D, k, i0, D, d.vec, u[k]);
      }
    } else if (!pre) {
#pragma unroll
      for (int k = 0; k < K; ++k) store8<TPR, SIDE>((IT*)a.r + row * d.D, k, i0, D, d.vec, u[k]);
    }
    if (pre) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(u[k][i], u[k][i], s[0]);
      row_sums<TPR, 1>(s, red, flip);
      const float rs = rsqrtf(s[0] * inv + d.eps);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        load_raw8<TPR, SIDE>(a.w_pre, k, i0, D, d.vec).get(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= u[k][i] * rs;
        store8<TPR, SIDE>((IT*)a.y + row * d.D, k, i0, D, d.vec, t);
      }
    }
    cur = next;
  }
}

}  // namespace

gdr_status resolve_norm(const gdr_norm_problem* p, NormDims* d) {
  if (p == nullptr || p->tokens < 0 || p->heads <= 0 || p->D <= 0) return GDR_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || !dtype_ok(p->res_dtype)) return GDR_ERR_INVALID_ARG;
  if (p->dtype == GDR_DTYPE_F32 && p->res_dtype != GDR_DTYPE_F32) return GDR_ERR_INVALID_ARG;
  if (!(p->eps > 0.f)) return GDR_ERR_INVALID_ARG;
  const long long w = (long long)p->heads * p->D;
  if ((p->ld_x != 0 && p->ld_x < w) || (p->ld_gate != 0 && p->ld_gate < w)) return GDR_ERR_INVALID_ARG;
  if (p->D > kNormMaxD || p->tokens > (1ll << 60) / w) return GDR_ERR_UNSUPPORTED;
  d->rows = p->tokens * p->heads;
  d->heads = p->heads;
  d->D = p->D;
  d->ld_x = p->ld_x ? p->ld_x : w;
  d->ld_gate = p->ld_gate ? p->ld_gate : w;
  if (d->ld_x == w && d->ld_gate == w) {  // heads without a gap are rows like any others
    d->heads = 1;
    d->ld_x = d->ld_gate = p->D;
  }
  d->eps = p->eps;
  d->vec = 0;
  return GDR_OK;
}

}  // namespace gdr

using namespace gdr;

extern "C" gdr_status gdr_norm_fwd(const gdr_norm_problem* p, const void* x, const float* w_post, const void* gate,
                                   const float* scale, const void* residual, const float* w_pre, void* r, void* y,
                                   gdr_stream_t stream) {
  NormDims d;
  const gdr_status st = resolve_norm(p, &d);
  if (st != GDR_OK) return st;
  if (d.rows == 0) return GDR_OK;  // tensors of no rows may have no address
  if (!w_post && !gate && !scale && !residual && !w_pre) return GDR_ERR_INVALID_ARG;
  if (w_pre && !residual && (w_post || gate || scale)) return GDR_ERR_INVALID_ARG;
  if ((!x || (w_pre && !y) || ((residual || !w_pre) && !r))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype), rel = residual ? dtype_bytes(p->res_dtype) : el;
  if (!elem_ok(x, el) || !elem_ok(gate, el) || !elem_ok(y, el) || !elem_ok(residual, rel) || !elem_ok(r, rel) ||
      !elem_ok(w_post, 4) || !elem_ok(scale, 4) || !elem_ok(w_pre, 4))
    return GDR_ERR_ALIGNMENT;
  d.vec = d.D % 8 == 0 && d.ld_x % 8 == 0 && d.ld_gate % 8 == 0 && vec_ok(x) && vec_ok(w_post) && vec_ok(gate) &&
          vec_ok(scale) && vec_ok(residual) && vec_ok(w_pre) && vec_ok(r) && vec_ok(y);
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  const FwdPtrs a{x, gate, residual, w_post, scale, w_pre, r, y};
  const int parts = (w_post ? kNormPost : 0) | (gate ? kNormGate : 0) | (scale ? kNormScale : 0) | (w_pre ? kNormPre : 0) |
                    (residual ? kNormRes : 0);
  auto go = [&](auto it, auto rt) {
    using IT = decltype(it);
    using RT = decltype(rt);
    return norm_shape(d.D, [&](auto tpr, auto k) {
      constexpr int TPR = decltype(tpr)::value, K = decltype(k)::value;
      return norm_parts(parts, [&](auto pt) {
        return norm_side<TPR>(d.vec, [&](auto side) {
          constexpr auto kernel = norm_fwd_kernel<IT, RT, TPR, K, decltype(pt)::value, decltype(side)::value>;
          static const long long most = (long long)kSmCount * resident_blocks(kernel, norm_block(TPR));
          const long long want = (d.rows + norm_rows(TPR) - 1) / norm_rows(TPR);
          kernel<<<(unsigned)(want < most ? want : most), norm_block(TPR), 0, s>>>(d, a);
          stage_mark(s, "norm_fwd");
          return cudaGetLastError();
        });
      });
    });
  };
  if (p->dtype == GDR_DTYPE_F32) return status_of(go(float{}, float{}));
  return status_of(p->res_dtype == GDR_DTYPE_F32 ? go(__nv_bfloat16{}, float{}) : go(__nv_bfloat16{}, __nv_bfloat16{}));
}
