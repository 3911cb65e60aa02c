// gdr_norm_bwd.cuh -- the block norms' backward kernel; gdr_norm_bwd_*.cu build it for their types.
#pragma once

#include "gdr_norm.cuh"

namespace gdr {

// Shared memory in which a thread's part of the next row waits, or 0.  Rows of one chunk per thread
// are loaded a row ahead into registers; of two chunks there is no room for that: gated rows and those of a
// residual add have the next row's copies under way here (4096 x 8192 bf16, backward: gated 101 -> 77 us, add 96 -> 75,
// 2048 x 8192 add in fp32 84 -> 79).  With everything the sums and weights of both norms already fill the
// registers and the shared memory's port, and it would cost (192 -> 230 us).
template <typename IT, typename RT, int TPR, int K, int PARTS, bool SIDE>
constexpr size_t norm_stage_bytes() {
  constexpr size_t chunk = (size_t)TPR * K, in = sizeof(Raw8<IT>), res = sizeof(Raw8<RT>);
  constexpr bool x = PARTS & (kNormPost | kNormGate | kNormScale), z = PARTS & kNormGate;
  constexpr bool pre = PARTS & kNormPre;
  constexpr size_t bytes = chunk * ((x ? in : 0) + (z ? in : 0) + (pre ? in + res : 0) + res);
  return TPR > 32 && K == 2 && !SIDE && PARTS >= 0 && !(x && pre) ? bytes : 0;
}

// Rows of more than a warp: the weights stay in shared memory (3 x D floats), since a row's work is
// a chain of two block sums and each read of a weight from the L2 would lengthen it (8192 x 4096
// with everything, fp32 stream: 193 us with global reads, 136 us with these).
template <typename IT, typename RT, int TPR, int K, int PARTS, bool SIDE>
__global__ void __launch_bounds__(norm_block(TPR)) norm_bwd_kernel(NormDims d, NormBwdPtrs a) {
  constexpr int kBlock = norm_block(TPR), kRows = norm_rows(TPR);
  constexpr bool kAhead = K == 1;  // two rows in registers; wider ones would spill
  constexpr bool kStage = norm_stage_bytes<IT, RT, TPR, K, PARTS, SIDE>() > 0;
  __shared__ float red[TPR > 32 ? 8 * TPR / 32 : 1];  // two buffers of 3 sums, two of 1
  __shared__ float cols[kRows > 1 ? kBlock * 8 : 1];
  int flip = 0, flip1 = 0;
  const bool post = PARTS >= 0 ? (PARTS & kNormPost) != 0 : a.w_post != nullptr;
  const bool gate = PARTS >= 0 ? (PARTS & kNormGate) != 0 : a.gate != nullptr;
  const bool scale = PARTS >= 0 ? (PARTS & kNormScale) != 0 : a.scale != nullptr;
  const bool pre = PARTS >= 0 ? (PARTS & kNormPre) != 0 : a.w_pre != nullptr;
  const bool has_dr = a.dr != nullptr;
  const bool need_x = post || gate || scale;
  const int i0 = threadIdx.x % TPR;
  const float inv = 1.f / (float)d.D;
  extern __shared__ __align__(16) float weights[];  // w_post, scale, w_pre, each of D rounded up to 8
  const int Dp = (d.D + 7) & ~7;
  if constexpr (TPR > 32) {
    for (int c = threadIdx.x; c < Dp; c += kBlock) {
      if (post) weights[c] = c < d.D ? a.w_post[c] : 0.f;
      if (scale) weights[Dp + c] = c < d.D ? a.scale[c] : 0.f;
      if (pre) weights[2 * Dp + c] = c < d.D ? a.w_pre[c] : 0.f;
    }
    __syncthreads();
  }
  auto weight = [&](const float* p, int part, int k, int D, float (&v)[8]) {
    if constexpr (TPR > 32)
      load_raw8<TPR, SIDE>(weights + part * Dp, k, i0, SIDE ? d.D : Dp, 1).get(v);
    else
      load_raw8<TPR, SIDE>(p, k, i0, D, d.vec).get(v);
  };
  constexpr int kAcc = PARTS >= 0 ? ((PARTS & kNormPost) != 0) + ((PARTS & kNormScale) != 0) + ((PARTS & kNormPre) != 0) : 3;
  constexpr int kScaleAt = PARTS >= 0 ? ((PARTS & kNormPost) != 0) : 1;
  constexpr int kPreAt = PARTS >= 0 ? ((PARTS & kNormPost) != 0) + ((PARTS & kNormScale) != 0) : 2;
  float acc[kAcc][K][8];  // sums over rows: dw_post, dscale, dw_pre as far as they are wanted
#pragma unroll
  for (int m = 0; m < kAcc; ++m)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[m][k][i] = 0.f;
  struct Row {
    Raw8<IT> x[K], z[K], dy[K];
    Raw8<RT> r[K], dr[K];
  };
  auto load = [&](long long row, Row& o) {
    const int D = row < d.rows ? d.D : 0;  // a missing row is zeros and is not stored
    const long long tok = token_of(d, row), at = (row - tok * d.heads) * d.D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (need_x) o.x[k] = load_raw8<TPR, SIDE>((const IT*)a.x + tok * d.ld_x + at, k, i0, D, d.vec);
      if (pre) {
        o.r[k] = load_raw8<TPR, SIDE>((const RT*)a.r + row * d.D, k, i0, D, d.vec);
        o.dy[k] = load_raw8<TPR, SIDE>((const IT*)a.dy + row * d.D, k, i0, D, d.vec);
      }
      if (has_dr) o.dr[k] = load_raw8<TPR, SIDE>((const RT*)a.dr + row * d.D, k, i0, D, d.vec);
      if (gate) o.z[k] = load_raw8<TPR, SIDE>((const IT*)a.gate + tok * d.ld_gate + at, k, i0, D, d.vec);
    }
  };
  // The same through shared memory: 16-byte pieces, each thread's own, in the order of load().  start: the
  // copies; else from there to o.
  auto staged = [&](long long row, Row& o, auto start) {
    uint4* slot = reinterpret_cast<uint4*>(weights + 3 * Dp) + i0;
    const long long tok = row / d.heads, at = (row - tok * d.heads) * d.D;
    auto move = [&](const auto* p, auto& raw, int k) {
      constexpr int kPieces = sizeof(raw) / 16;
      const int c = channel<TPR, SIDE>(k, i0, 0);
#pragma unroll
      for (int i = 0; i < kPieces; ++i, slot += TPR)
        if constexpr (decltype(start)::value)
          copy_async<16>(slot, c < d.D ? reinterpret_cast<const uint4*>(p + c) + i : reinterpret_cast<const uint4*>(p), c < d.D ? 16 : 0);
        else
          reinterpret_cast<uint4*>(&raw)[i] = *slot;
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (need_x) move((const IT*)a.x + tok * d.ld_x + at, o.x[k], k);
      if (pre) {
        move((const RT*)a.r + row * d.D, o.r[k], k);
        move((const IT*)a.dy + row * d.D, o.dy[k], k);
      }
      if (has_dr) move((const RT*)a.dr + row * d.D, o.dr[k], k);
      if (gate) move((const IT*)a.gate + tok * d.ld_gate + at, o.z[k], k);
    }
  };
  const long long step = (long long)gridDim.x * kRows;
  long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  Row cur;
  if (kAhead) load(row, cur);
  if (kStage && row < d.rows) staged(row, cur, std::true_type{});
  for (long long base = (long long)blockIdx.x * kRows; base < d.rows; base += step, row += step) {
    Row next;
    if (kStage) {
      copy_async_wait();
      staged(row, cur, std::false_type{});
    } else if (!kAhead) {
      load(row, cur);
    }
    if (kAhead && base + step < d.rows) load(row + step, next);
    const int D = row < d.rows ? d.D : 0;
    float du[K][8], t[8], v[8], w[8];
    float s[3] = {0.f, 0.f, 0.f};  // sum x^2, sum r^2, sum dy w_pre r
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (post) {
        cur.x[k].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(v[i], v[i], s[0]);
      }
      if (pre) {
        cur.r[k].get(v);
        cur.dy[k].get(t);
        weight(a.w_pre, 2, k, D, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[1] = fmaf(v[i], v[i], s[1]);
          s[2] = fmaf(t[i] * w[i], v[i], s[2]);
        }
      }
    }
    if (post || pre) row_sums<TPR, 3>(s, red, flip);
    if (kStage && base + step < d.rows) staged(row + step, cur, std::true_type{});  // behind the sums' barrier: the slots are read
    const float rx = post ? rsqrtf(s[0] * inv + d.eps) : 1.f;
    const float rr = rsqrtf(s[1] * inv + d.eps), m1 = s[2] * inv * rr;  // m1: mean(t rh)
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (has_dr) {
        cur.dr[k].get(du[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) du[k][i] = 0.f;
      }
      if (pre) {
        cur.r[k].get(v);
        cur.dy[k].get(t);
        weight(a.w_pre, 2, k, D, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float rh = v[i] * rr;
          acc[kPreAt < kAcc ? kPreAt : 0][k][i] = fmaf(t[i], rh, acc[kPreAt < kAcc ? kPreAt : 0][k][i]);
          du[k][i] = fmaf(rr, t[i] * w[i] - rh * m1, du[k][i]);
        }
      }
      if (a.dres) store8<TPR, SIDE>((RT*)a.dres + row * d.D, k, i0, D, d.vec, du[k]);
      if (need_x) {
        float sc[8], z[8];
        cur.x[k].get(v);
        if (post) weight(a.w_post, 0, k, D, w);
        if (scale) weight(a.scale, 1, k, D, sc);
        if (gate) cur.z[k].get(z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = v[i] * rx;
          const float n = post ? xh * w[i] : xh;
          float e = du[k][i], act = 1.f;
          if (gate) {
            const float sg = sigmoid_f(z[i]);
            act = z[i] * sg;
            t[i] = (scale ? e * sc[i] : e) * n * (sg * fmaf(z[i], 1.f - sg, 1.f));
          }
          if (scale) {
            acc[kScaleAt < kAcc ? kScaleAt : 0][k][i] = fmaf(e, n * act, acc[kScaleAt < kAcc ? kScaleAt : 0][k][i]);
            e *= sc[i];
          }
          if (gate) e *= act;
          if (post) {
            acc[0][k][i] = fmaf(e, xh, acc[0][k][i]);
            e *= w[i];
            q[0] = fmaf(e, xh, q[0]);
          }
          du[k][i] = e;
        }
        if (gate) store8<TPR, SIDE>((IT*)a.dgate + row * d.D, k, i0, D, d.vec, t);
      }
    }
    if (post) {
      row_sums<TPR, 1>(q, red + (TPR > 32 ? 6 * TPR / 32 : 0), flip1);
      const float m2 = q[0] * inv * rx;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        cur.x[k].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) du[k][i] = rx * (du[k][i] - v[i] * m2);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) store8<TPR, SIDE>((IT*)a.dx + row * d.D, k, i0, D, d.vec, du[k]);
    if (kAhead) cur = next;
  }
#pragma unroll
  for (int m = 0; m < kAcc; ++m) {
    const int slot = PARTS < 0 ? m : m == kPreAt && (PARTS & kNormPre) ? 2 : m == kScaleAt && (PARTS & kNormScale) ? 1 : 0;
    float* out = a.partial + ((long long)blockIdx.x * 3 + slot) * d.D;
    if constexpr (kRows == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) store8<TPR, SIDE>(out, k, i0, d.D, d.vec, acc[m][k]);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) cols[threadIdx.x * 8 + i] = acc[m][k][i];
        __syncthreads();
        for (int j = threadIdx.x; j < TPR * 8; j += kBlock) {
          float sum = 0.f;
#pragma unroll 4
          for (int rw = 0; rw < kRows; ++rw) sum += cols[rw * TPR * 8 + j];
          if (8 * k * TPR + j < d.D) out[8 * k * TPR + j] = sum;
        }
      }
    }
  }
}

template <typename IT, typename RT>
cudaError_t norm_bwd_launch(const NormDims& d, const NormBwdPtrs& a, int parts, long long* grid, cudaStream_t s) {
  return norm_shape(d.D, [&](auto tpr, auto k) {
    constexpr int TPR = decltype(tpr)::value, K = decltype(k)::value;
    return norm_parts(parts, [&](auto pt) {
      return norm_side<TPR>(d.vec, [&](auto side) {
        constexpr auto kernel = norm_bwd_kernel<IT, RT, TPR, K, decltype(pt)::value, decltype(side)::value>;
        constexpr size_t stage = norm_stage_bytes<IT, RT, TPR, K, decltype(pt)::value, decltype(side)::value>();
        constexpr size_t widest = TPR > 32 ? 3 * sizeof(float) * 8 * TPR * K + stage : 0;  // for the shape's widest row
        const size_t smem = TPR > 32 ? 3 * sizeof(float) * (size_t)((d.D + 7) & ~7) + stage : 0;
        static_assert(widest + 1024 <= 227 * 1024, "shared memory of a block");
        if (smem > 0) {
          const cudaError_t e = set_smem_once((const void*)kernel, widest);
          if (e != cudaSuccess) return e;
        }
        static const long long most = (long long)kSmCount * resident_blocks(kernel, norm_block(TPR), widest);
        if (*grid > most) *grid = most;
        kernel<<<(unsigned)*grid, norm_block(TPR), smem, s>>>(d, a);
        stage_mark(s, "norm_bwd");
        return cudaGetLastError();
      });
    });
  });
}

}  // namespace gdr
