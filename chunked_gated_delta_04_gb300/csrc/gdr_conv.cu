// gdr_conv.cu -- the short causal depthwise convolution of a mixer's inputs (include/gdr_block.h):
//
//   pre[t, c] = bias[c] + sum_{j < W} w[c, j] X[t - (W - 1) + j, c],     y = silu(pre) or pre,
//
// X = the sequence's tokens preceded by W - 1 rows of state, and its backward
//
//   dpre = dy act'(pre),   dX[s] = sum_j w[j] dpre[s + (W - 1) - j],
//   dw[j] = sum_t dpre[t] X[t - (W - 1) + j],   dbias = sum_t dpre[t].
//
// Both are bound by memory: 2 W multiply-adds per element against 4 (forward) or 6 (backward)
// bytes in bf16.  A thread owns V channels (16 bytes) and walks a run of tokens with the last
// W - 1 inputs (and, backward, the last W - 1 dpre) in registers, so each element is read once but
// for the W - 1 rows in front of (backward: also behind) a run, which its neighbour's reads have
// brought into the L2.
#include "gdr_block.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;

struct ConvDims {
  int T, C, num_seqs, silu;
  long long total, ld_x, ld_dy;
  const int32_t* cu;
  const uint32_t* status;  // variable length: the sequence check's word
};

// The sequence [s0, s1) that contains token t, and the ones after it.
struct SeqWalk {
  int n;
  long long s0, s1;
  __device__ void find(const ConvDims& d, long long t) {
    if (d.cu) {
      n = seq_of(d.cu, d.num_seqs, t);
      s0 = d.cu[n];
      s1 = d.cu[n + 1];
    } else {
      n = (int)(t / d.T);
      s0 = (long long)n * d.T;
      s1 = s0 + d.T;
    }
  }
  __device__ void next(const ConvDims& d) {  // empty sequences are passed over
    do {
      ++n;
      s0 = s1;
      s1 = d.cu ? d.cu[n + 1] : s1 + d.T;
    } while (s1 == s0);
  }
  __device__ void of(const ConvDims& d, int seq) {
    n = seq;
    s0 = d.cu ? d.cu[n] : (long long)n * d.T;
    s1 = d.cu ? d.cu[n + 1] : s0 + d.T;
  }
};

template <int V, int W>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, long long c, float (&wt)[W][V],
                                          float (&b)[V]) {
  if constexpr (V > 1 && W == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(w + (c + i) * 4);
      wt[0][i] = x.x; wt[1][i] = x.y; wt[2][i] = x.z; wt[3][i] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) wt[j][i] = w[(c + i) * W + j];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = bias ? bias[c + i] : 0.f;
}

// Row p (p < s1) of X: a token, or, before s0, a row of the state.
template <typename IT, int V, int W>
__device__ __forceinline__ void load_row(const ConvDims& d, const SeqWalk& q, const IT* x, const IT* state,
                                         long long p, long long c, float (&v)[V]) {
  if (p >= q.s0) {
    load_v<V>(x + p * d.ld_x + c, v);
  } else if (state) {
    load_v<V>(state + ((long long)q.n * (W - 1) + (p - q.s0 + W - 1)) * d.C + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
  }
}

template <int V, int W>
__device__ __forceinline__ void taps(const float (&win)[W][V], const float (&wt)[W][V], const float (&b)[V],
                                     float (&pre)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) pre[i] = b[i];
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) pre[i] = fmaf(wt[j][i], win[j][i], pre[i]);
}

template <typename IT, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvDims d, const IT* __restrict__ x,
                                                            const float* __restrict__ w,
                                                            const float* __restrict__ bias,
                                                            const IT* __restrict__ state, IT* __restrict__ y,
                                                            IT* __restrict__ last, int L) {
  if (d.status && *d.status) return;
  const int ncg = d.C / V;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long runs = (d.total + L - 1) / L, run = id / ncg;
  const long long c = (id - run * ncg) * V;
  SeqWalk q;
  if (run >= runs) {  // the state after the last token: one thread per sequence and V channels
    if (last == nullptr || run - runs >= d.num_seqs) return;
    q.of(d, (int)(run - runs));
    float v[V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      load_row<IT, V, W>(d, q, x, state, q.s1 - (W - 1) + j, c, v);
      store_v<V>(last + ((long long)q.n * (W - 1) + j) * d.C + c, v);
    }
    return;
  }
  const long long t0 = run * L, t1 = min(t0 + L, d.total);
  float wt[W][V], b[V], win[W][V], pre[V];
  load_taps<V, W>(w, bias, c, wt, b);
  q.find(d, t0);
  for (long long t = t0; t < t1;) {
    const long long end = min(t1, q.s1);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<IT, V, W>(d, q, x, state, t - (W - 1) + j, c, win[j + 1]);
    auto one = [&](long long p, const float (&in)[V]) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
      for (int i = 0; i < V; ++i) win[W - 1][i] = in[i];
      taps<V, W>(win, wt, b, pre);
      if (d.silu) {
#pragma unroll
        for (int i = 0; i < V; ++i) pre[i] *= sigmoid_f(pre[i]);
      }
      store_v<V>(y + p * d.C + c, pre);
    };
    for (; t + 4 <= end; t += 4) {  // four rows in flight
      float in[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) load_v<V>(x + (t + u) * d.ld_x + c, in[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) one(t + u, in[u]);
    }
    for (; t < end; ++t) {
      float in[V];
      load_v<V>(x + t * d.ld_x + c, in);
      one(t, in);
    }
    if (t < t1) q.next(d);
  }
}

// dpre of token t from its window and dy.
template <int V, int W>
__device__ __forceinline__ void grad_pre(const float (&win)[W][V], const float (&wt)[W][V], const float (&b)[V],
                                         int silu, float (&g)[V]) {
  if (silu) {
    float pre[V];
    taps<V, W>(win, wt, b, pre);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = sigmoid_f(pre[i]);
      g[i] *= s * fmaf(pre[i], 1.f - s, 1.f);
    }
  }
}

// Blocks of kThreads / cpb runs of L tokens by cpb groups of V channels; a block's sums of dw and
// dbias go to partial[blockIdx.x][W + 1][C].  blockIdx.x >= tiles: dstate, one sequence per run.
template <typename IT, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvDims d, const IT* __restrict__ x,
                                                            const float* __restrict__ w,
                                                            const float* __restrict__ bias,
                                                            const IT* __restrict__ state,
                                                            const IT* __restrict__ dy,
                                                            const IT* __restrict__ dlast, IT* __restrict__ dx,
                                                            IT* __restrict__ dstate, float* __restrict__ partial,
                                                            int L, int cpb, int tiles) {
  __shared__ float red[kThreads * V];
  if (d.status && *d.status) return;
  const int subs = kThreads / cpb, sub = threadIdx.x / cpb, cg = threadIdx.x - sub * cpb;
  const long long c = ((long long)blockIdx.y * cpb + cg) * V;
  const bool live = c < d.C;
  SeqWalk q;
  float wt[W][V], b[V], win[W][V], dwin[W][V], g[V];
  float acc[W + 1][V];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
  if (live) load_taps<V, W>(w, bias, c, wt, b);

  // dX of row p of sequence q from the dpre of rows p .. p + W - 1 (dwin[j] = dpre[p + j])
  auto row_grad = [&](long long p, float (&out)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = fmaf(wt[W - 1 - j][i], dwin[j][i], out[i]);
    const long long k = p - (q.s1 - (W - 1));
    if (dlast && k >= 0) {
      float v[V];
      load_v<V>(dlast + ((long long)q.n * (W - 1) + k) * d.C + c, v);
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] += v[i];
    }
  };
  auto push = [&](float (&ring)[W][V], const float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) ring[j][i] = ring[j + 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) ring[W - 1][i] = v[i];
  };
  // dpre of row u of sequence q, both windows moved on to it
  auto advance = [&](long long u, const float (&in)[V], float (&dyv)[V]) {
    push(win, in);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = dyv[i];
    grad_pre<V, W>(win, wt, b, d.silu, g);
    push(dwin, g);
  };
  auto open = [&](long long u) {  // windows in front of row u; dpre before it counts as zero
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<IT, V, W>(d, q, x, state, u - (W - 1) + j, c, win[j + 1]);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) dwin[j][i] = 0.f;
  };
  const float zero[V] = {};

  if ((int)blockIdx.x >= tiles) {
    const long long n = (long long)(blockIdx.x - tiles) * subs + sub;
    if (!live || n >= d.num_seqs) return;
    q.of(d, (int)n);
    open(q.s0);
    for (int k = 0; k < W - 1; ++k) {  // row u = s0 + k completes the window of row u - (W - 1)
      const long long u = q.s0 + k;
      if (u < q.s1) {
        float in[V], dyv[V];
        load_v<V>(x + u * d.ld_x + c, in);
        load_v<V>(dy + u * d.ld_dy + c, dyv);
        advance(u, in, dyv);
      } else {
        push(dwin, zero);
      }
      // state row k is X row s0 - (W - 1) + k: dpre of rows s0 .. s0 + k reach it
      float out[V];
      row_grad(u - (W - 1), out);
      store_v<V>(dstate + (n * (W - 1) + k) * d.C + c, out);
    }
    return;
  }

  const long long t0 = ((long long)blockIdx.x * subs + sub) * L, t1 = min(t0 + L, d.total);
  if (live && t0 < t1) {
    q.find(d, t0);
    for (long long a = t0; a < t1;) {
      const long long end = min(t1, q.s1);          // rows [a, end) are this run's
      const long long stop = min(q.s1, end + W - 1);  // dpre is needed up to here
      open(a);
      auto emit = [&](long long u) {  // row u's dpre is in: row u - (W - 1) is complete
        const long long p = u - (W - 1);
        if (p >= a && p < end) {
          float out[V];
          row_grad(p, out);
          store_v<V>(dx + p * d.C + c, out);
        }
      };
      auto one = [&](long long u, const float (&in)[V], float (&dyv)[V]) {
        advance(u, in, dyv);
        if (u < end) {
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[j][i] = fmaf(g[i], win[j][i], acc[j][i]);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[W][i] += g[i];
        }
        emit(u);
      };
      long long u = a;
      for (; u + 4 <= stop; u += 4) {
        float in[4][V], dyv[4][V];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          load_v<V>(x + (u + k) * d.ld_x + c, in[k]);
          load_v<V>(dy + (u + k) * d.ld_dy + c, dyv[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) one(u + k, in[k], dyv[k]);
      }
      for (; u < stop; ++u) {
        float in[V], dyv[V];
        load_v<V>(x + u * d.ld_x + c, in);
        load_v<V>(dy + u * d.ld_dy + c, dyv);
        one(u, in, dyv);
      }
      for (; u < end + W - 1; ++u) {  // past the sequence's end: no dpre
        push(dwin, zero);
        emit(u);
      }
      a = end;
      if (a < t1) q.next(d);
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) red[(sub * V + i) * cpb + cg] = acc[j][i];
    __syncthreads();
    for (int k = threadIdx.x; k < cpb * V; k += kThreads) {
      const int i = k / cpb, kg = k - i * cpb;
      float a = 0.f;
      for (int r = 0; r < subs; ++r) a += red[(r * V + i) * cpb + kg];
      const long long cc = ((long long)blockIdx.y * cpb + kg) * V + i;
      if (cc < d.C) partial[((long long)blockIdx.x * (W + 1) + j) * d.C + cc] = a;
    }
  }
}

template <typename IT, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(int B, int C, long long ld_x, int silu, int num_slots,
                                                             const IT* __restrict__ x, const float* __restrict__ w,
                                                             const float* __restrict__ bias, IT* __restrict__ pool,
                                                             const int32_t* __restrict__ slots,
                                                             IT* __restrict__ y) {
  const int ncg = C / V;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x, b = id / ncg;
  if (b >= B) return;
  const long long c = (id - b * ncg) * V;
  const long long slot = slots ? slots[b] : b;
  float pre[V];
  if (slot < 0 || slot >= num_slots) {
#pragma unroll
    for (int i = 0; i < V; ++i) pre[i] = 0.f;
    store_v<V>(y + b * C + c, pre);
    return;
  }
  IT* st = pool + slot * (W - 1) * C + c;
  float win[W][V], wt[W][V], bs[V];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_v<V>(st + (long long)j * C, win[j]);
  load_v<V>(x + b * ld_x + c, win[W - 1]);
  load_taps<V, W>(w, bias, c, wt, bs);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_v<V>(st + (long long)j * C, win[j + 1]);
  taps<V, W>(win, wt, bs, pre);
  if (silu) {
#pragma unroll
    for (int i = 0; i < V; ++i) pre[i] *= sigmoid_f(pre[i]);
  }
  store_v<V>(y + b * C + c, pre);
}

gdr_status resolve_conv(const gdr_conv_problem* p, bool step, ConvDims* d) {
  if (p == nullptr || p->B < 0 || p->T < 0 || p->C <= 0 || p->num_seqs < 0) return GDR_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || (p->silu != 0 && p->silu != 1)) return GDR_ERR_INVALID_ARG;
  if ((p->ld_x != 0 && p->ld_x < p->C) || (p->ld_dy != 0 && p->ld_dy < p->C)) return GDR_ERR_INVALID_ARG;
  if (step) {
    if (p->T != 1 || p->cu_seqlens || p->num_slots < 0) return GDR_ERR_INVALID_ARG;
  } else if (p->cu_seqlens ? p->B != 1 || p->num_seqs < 1 : p->num_seqs != p->B) {
    return GDR_ERR_INVALID_ARG;
  }
  if (p->W < 2 || p->W > 4) return GDR_ERR_UNSUPPORTED;
  if ((long long)p->B * p->T >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  d->T = p->T;
  d->C = p->C;
  d->num_seqs = p->num_seqs;
  d->silu = p->silu;
  d->total = (long long)p->B * p->T;
  d->ld_x = p->ld_x ? p->ld_x : p->C;
  d->ld_dy = p->ld_dy ? p->ld_dy : p->C;
  d->cu = p->cu_seqlens;
  d->status = nullptr;
  return GDR_OK;
}

// Launch shape of the backward: channel groups per block and tokens per run.
struct BwdShape {
  int cpb, L;
  long long tiles;
};
BwdShape bwd_shape(const ConvDims& d) {
  BwdShape b;
  const int ncg = (d.C + 7) / 8;
  b.cpb = ncg >= 32 ? 32 : ncg >= 16 ? 16 : 8;
  const int subs = kThreads / b.cpb;
  b.L = 32;
  while (b.L > 4 && (d.total + b.L * subs - 1) / (b.L * subs) * ((ncg + b.cpb - 1) / b.cpb) < 2 * kSmCount) b.L /= 2;
  b.tiles = (d.total + (long long)b.L * subs - 1) / ((long long)b.L * subs);
  return b;
}

size_t conv_bwd_bytes(const ConvDims& d, int W) {
  return 256 + block_align(sizeof(float) * (size_t)bwd_shape(d).tiles * (W + 1) * d.C);
}

template <typename F>
cudaError_t by_type(gdr_dtype dt, bool vec, int W, F f) {
  auto width = [&](auto it, auto v) {
    return W == 2 ? f(it, v, std::integral_constant<int, 2>{})
                  : W == 3 ? f(it, v, std::integral_constant<int, 3>{}) : f(it, v, std::integral_constant<int, 4>{});
  };
  using V8 = std::integral_constant<int, 8>;
  using V1 = std::integral_constant<int, 1>;
  if (dt == GDR_DTYPE_BF16) return vec ? width(__nv_bfloat16{}, V8{}) : width(__nv_bfloat16{}, V1{});
  return vec ? width(float{}, V8{}) : width(float{}, V1{});
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_conv_fwd_workspace_bytes(const gdr_conv_problem* p) {
  ConvDims d;
  return resolve_conv(p, false, &d) == GDR_OK && d.cu ? 256 : 0;
}

size_t gdr_conv_bwd_workspace_bytes(const gdr_conv_problem* p) {
  ConvDims d;
  return resolve_conv(p, false, &d) == GDR_OK ? conv_bwd_bytes(d, p->W) : 0;
}

gdr_status gdr_conv_fwd(const gdr_conv_problem* p, const void* x, const float* w, const float* bias,
                        const void* state, void* y, void* last, void* workspace, size_t workspace_bytes,
                        gdr_stream_t stream) {
  ConvDims d;
  const gdr_status st = resolve_conv(p, false, &d);
  if (st != GDR_OK) return st;
  if (!w || (d.total > 0 && (!x || !y))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(x, el) || !elem_ok(y, el) || !elem_ok(state, el) || !elem_ok(last, el) || !elem_ok(w, 4) ||
      !elem_ok(bias, 4) || !elem_ok(d.cu, 4) || ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  if (d.cu && (!workspace || workspace_bytes < 256)) return GDR_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  if (d.cu) {
    d.status = (const uint32_t*)workspace;
    const cudaError_t e = launch_seq_check(d.cu, d.num_seqs, d.T, (uint32_t*)workspace, s);
    if (e != cudaSuccess) return status_of(e);
  }
  const bool vec = d.C % 8 == 0 && d.ld_x % 8 == 0 && vec_ok(x) && vec_ok(y) && vec_ok(state) && vec_ok(last) && vec_ok(w);
  const long long ncg = vec ? d.C / 8 : d.C;
  // runs of 32 tokens read 3 rows twice (from the L2); short batches take shorter runs so that
  // there are threads enough to keep the memory busy
  int L = 32;
  while (L > 4 && (d.total + L - 1) / L * ncg < (long long)kSmCount * 1024) L /= 2;
  const long long threads = ((d.total + L - 1) / L + (last ? d.num_seqs : 0)) * ncg;
  if (threads == 0) return GDR_OK;
  const long long grid = (threads + kThreads - 1) / kThreads;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  return status_of(by_type(p->dtype, vec, p->W, [&](auto it, auto v, auto wd) {
    using IT = decltype(it);
    conv_fwd_kernel<IT, decltype(v)::value, decltype(wd)::value><<<(unsigned)grid, kThreads, 0, s>>>(
        d, (const IT*)x, w, bias, (const IT*)state, (IT*)y, (IT*)last, L);
    stage_mark(s, "conv_fwd");
    return cudaGetLastError();
  }));
}

gdr_status gdr_conv_bwd(const gdr_conv_problem* p, const void* x, const float* w, const float* bias,
                        const void* state, const void* dy, const void* dlast, void* dx, float* dw, float* dbias,
                        void* dstate, void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  ConvDims d;
  const gdr_status st = resolve_conv(p, false, &d);
  if (st != GDR_OK) return st;
  if (!w || !dw || (d.total > 0 && (!x || !dy || !dx))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(x, el) || !elem_ok(dy, el) || !elem_ok(dx, el) || !elem_ok(state, el) || !elem_ok(dlast, el) ||
      !elem_ok(dstate, el) || !elem_ok(w, 4) || !elem_ok(bias, 4) || !elem_ok(dw, 4) || !elem_ok(dbias, 4) ||
      !elem_ok(d.cu, 4) || ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < conv_bwd_bytes(d, p->W)) return GDR_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  if (d.cu) {
    d.status = (const uint32_t*)workspace;
    const cudaError_t e = launch_seq_check(d.cu, d.num_seqs, d.T, (uint32_t*)workspace, s);
    if (e != cudaSuccess) return status_of(e);
  }
  float* partial = (float*)((char*)workspace + 256);
  const bool vec = d.C % 8 == 0 && d.ld_x % 8 == 0 && d.ld_dy % 8 == 0 && vec_ok(x) && vec_ok(dy) && vec_ok(dx) &&
                   vec_ok(state) && vec_ok(dlast) && vec_ok(dstate) && vec_ok(w);
  const BwdShape b = bwd_shape(d);
  const int subs = kThreads / b.cpb;
  const long long gx = b.tiles + (dstate ? ((long long)d.num_seqs + subs - 1) / subs : 0);
  const int ncg = vec ? d.C / 8 : d.C;
  const int gy = (ncg + b.cpb - 1) / b.cpb;
  if (gx >= (1ll << 31) || gy > 65535) return GDR_ERR_UNSUPPORTED;
  if (gx > 0) {
    const cudaError_t e = by_type(p->dtype, vec, p->W, [&](auto it, auto v, auto wd) {
      using IT = decltype(it);
      conv_bwd_kernel<IT, decltype(v)::value, decltype(wd)::value><<<dim3((unsigned)gx, gy), kThreads, 0, s>>>(
          d, (const IT*)x, w, bias, (const IT*)state, (const IT*)dy, (const IT*)dlast, (IT*)dx, (IT*)dstate, partial,
          b.L, b.cpb, (int)b.tiles);
      stage_mark(s, "conv_bwd");
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return status_of(e);
  }
  ColumnSums out = {};
  out.mat = dw;
  out.mat_parts = p->W;
  out.vec[0] = dbias;
  out.parts = p->W + 1;
  out.width = d.C;
  out.status = d.status;
  return status_of(launch_column_sums(partial, b.tiles, out, s, "conv_dw"));
}

gdr_status gdr_conv_step(const gdr_conv_problem* p, const void* x, const float* w, const float* bias, void* pool,
                         const int32_t* slots, void* y, gdr_stream_t stream) {
  ConvDims d;
  const gdr_status st = resolve_conv(p, true, &d);
  if (st != GDR_OK) return st;
  if (d.total > 0 && (!w || !x || !y || (!pool && p->num_slots > 0))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(x, el) || !elem_ok(y, el) || !elem_ok(pool, el) || !elem_ok(w, 4) || !elem_ok(bias, 4) ||
      !elem_ok(slots, 4))
    return GDR_ERR_ALIGNMENT;
  if (d.total == 0) return GDR_OK;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  const bool vec = d.C % 8 == 0 && d.ld_x % 8 == 0 && vec_ok(x) && vec_ok(y) && vec_ok(pool) && vec_ok(w);
  const long long grid = (d.total * (vec ? d.C / 8 : d.C) + kThreads - 1) / kThreads;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  return status_of(by_type(p->dtype, vec, p->W, [&](auto it, auto v, auto wd) {
    using IT = decltype(it);
    conv_step_kernel<IT, decltype(v)::value, decltype(wd)::value><<<(unsigned)grid, kThreads, 0, s>>>(
        p->B, d.C, d.ld_x, d.silu, p->num_slots, (const IT*)x, w, bias, (IT*)pool, slots, (IT*)y);
    stage_mark(s, "conv_step");
    return cudaGetLastError();
  }));
}

}  // extern "C"
