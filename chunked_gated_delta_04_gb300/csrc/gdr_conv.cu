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
// bytes in bf16.  A thread owns V channels and walks a run of tokens with the last
// W - 1 inputs (and, backward, the last W - 1 dpre) in registers, so each element is read once but
// for the W - 1 rows in front of (backward: also behind) a run, which its neighbour's reads have
// brought into the L2.
#include <initializer_list>

#include "gdr_block.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;        // channels per thread of the vector paths
constexpr int kFwdBlocks = 3;  // blocks per SM of the forward

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

// V channels of a row as P register pairs (V = 1: the upper half of the pair is idle).
template <int V>
constexpr int kPairs = (V + 1) / 2;

template <int V, int W>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, long long c, f32x2 (&wt)[W][kPairs<V>],
                                          f32x2 (&b)[kPairs<V>]) {
  float t[W][kPairs<V> * 2] = {}, bs[kPairs<V> * 2] = {};
  if constexpr (V > 1 && W == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(w + (c + i) * 4);
      t[0][i] = x.x; t[1][i] = x.y; t[2][i] = x.z; t[3][i] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) t[j][i] = w[(c + i) * W + j];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) bs[i] = bias ? bias[c + i] : 0.f;
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
    b[i] = pack2(bs[2 * i], bs[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j][i] = pack2(t[j][2 * i], t[j][2 * i + 1]);
  }
}

// V neighbouring elements as they come from memory, converted where they are used, so that a load is
// not waited for before that.  Aligned to its size: in shared memory it is the target of one asynchronous copy.
template <typename IT, int V>
struct alignas(V * sizeof(IT)) Raw {
  uint32_t w[V * sizeof(IT) / 4];
  __device__ __forceinline__ void load(const IT* p) {
    if constexpr (sizeof(w) == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < (int)(sizeof(w) / 4); i += 4) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void get(f32x2 (&v)[kPairs<V>]) const {
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
      if constexpr (sizeof(IT) == 4)
        v[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else
        v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
};
template <typename IT>
struct Raw<IT, 1> {
  IT w;
  __device__ __forceinline__ void load(const IT* p) { w = *p; }
  __device__ __forceinline__ void get(f32x2 (&v)[1]) const { v[0] = pack2(to_f32(w), 0.f); }
};
template <int V, typename IT>
__device__ __forceinline__ void store_row(IT* p, const f32x2 (&v)[kPairs<V>]) {
  float f[kPairs<V> * 2];
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
    f[2 * i] = lo2(v[i]);
    f[2 * i + 1] = hi2(v[i]);
  }
  store_v<V>(p, *reinterpret_cast<const float(*)[V]>(&f));
}

// Calls row(t, in) for the n rows of NS tensors in order, in[s] being the row's V channels of tensor s.
// Vector rows are copied, DEEP - 1 of them ahead, to slots in shared memory that only this thread uses
// (slots: its column of [DEEP][NS][kThreads]), so that the rows in flight take no registers; a slot is
// refilled a step after it was read.  Scalar rows wait in registers, four ahead.  Bytes in flight are
// what a kernel's nearness to the memory rate depends on: forward, B = 2, T = 4096, C = 6144, bf16, from
// a cold L2: 46 us with four rows in registers, 43 us with seven in shared memory.
// Groups of four rows run without conditions on what row() keeps: its windows' moves are renamings.
template <typename IT, int V, int NS, int DEEP, typename F>
__device__ __forceinline__ void walk_rows(const IT* const (&src)[NS], const long long (&ld)[NS], int n, Raw<IT, V>* slots,
                                          F row) {
  static_assert(alignof(Raw<IT, V>) == sizeof(Raw<IT, V>), "a slot takes one copy of its size");
  const IT* p[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) p[s] = src[s];
  if constexpr (V > 1) {
    auto start = [&](int slot, bool some) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (some) copy_async<sizeof(Raw<IT, V>)>(slots + (slot * NS + s) * kThreads, p[s], sizeof(Raw<IT, V>));
        p[s] += ld[s];
      }
      copy_async_commit();
    };
#pragma unroll
    for (int i = 0; i < DEEP - 1; ++i) start(i, i < n);
    auto step = [&](int t) {
      copy_async_wait_group<DEEP - 2>();  // of the t + DEEP - 1 rows started, row t is there
      f32x2 in[NS][kPairs<V>];
#pragma unroll
      for (int s = 0; s < NS; ++s) slots[(t % DEEP * NS + s) * kThreads].get(in[s]);
      start((t + DEEP - 1) % DEEP, t + DEEP - 1 < n);
      row(t, in);
    };
    int t = 0;
    for (; t + 4 <= n; t += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) step(t + u);
    }
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (t + u < n) step(t + u);
  } else {
    Raw<IT, V> r[4][NS];
    auto start = [&](int i, bool some) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (some) r[i][s].load(p[s]);
        p[s] += ld[s];
      }
    };
    auto step = [&](int t, int u) {
      f32x2 in[NS][kPairs<V>];
#pragma unroll
      for (int s = 0; s < NS; ++s) r[u][s].get(in[s]);
      start(u, t + 4 < n);
      row(t, in);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) start(i, i < n);
    int t = 0;
    for (; t + 4 <= n; t += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) step(t + u, u);
    }
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (t + u < n) step(t + u, u);
  }
}

// Row p (p < s1) of X: a token, or, before s0, a row of the state.
template <typename IT, int V, int W>
__device__ __forceinline__ void load_row(const ConvDims& d, const SeqWalk& q, const IT* x, const IT* state,
                                         long long p, long long c, f32x2 (&v)[kPairs<V>]) {
  Raw<IT, V> r;
  if (p >= q.s0) {
    r.load(x + p * d.ld_x + c);
    r.get(v);
  } else if (state) {
    r.load(state + ((long long)q.n * (W - 1) + (p - q.s0 + W - 1)) * d.C + c);
    r.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) v[i] = 0;
  }
}

template <int V, int W>
__device__ __forceinline__ void taps(const f32x2 (&win)[W][kPairs<V>], const f32x2 (&wt)[W][kPairs<V>],
                                     const f32x2 (&b)[kPairs<V>], f32x2 (&pre)[kPairs<V>]) {
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) pre[i] = b[i];
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) pre[i] = fma2(wt[j][i], win[j][i], pre[i]);
}
template <int V>
__device__ __forceinline__ void silu_row(f32x2 (&v)[kPairs<V>]) {
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) v[i] = mul2(v[i], sigmoid2(v[i]));
}
// The window moves on by one row.
template <int V, int W>
__device__ __forceinline__ void push(f32x2 (&ring)[W][kPairs<V>], const f32x2 (&v)[kPairs<V>]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) ring[j][i] = ring[j + 1][i];
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) ring[W - 1][i] = v[i];
}

// B = 2, T = 4096, C = 6144, bf16, W = 4, from a cold L2: 43 us, 201 MB, 4.7 TB/s.  Runs of 32 tokens
// (2.5 waves) instead of one wave's cost 6 us.
template <typename IT, int V, int W>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) conv_fwd_kernel(ConvDims d, const IT* __restrict__ x,
                                                               const float* __restrict__ w,
                                                               const float* __restrict__ bias,
                                                               const IT* __restrict__ state, IT* __restrict__ y,
                                                               IT* __restrict__ last, int L) {
  constexpr int P = kPairs<V>, kDeep = 8;
  __shared__ Raw<IT, V> slots[V > 1 ? kDeep * kThreads : 1];
  if (d.status && *d.status) return;
  const int ncg = d.C / V;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long runs = (d.total + L - 1) / L, run = id / ncg;
  const long long c = (id - run * ncg) * V;
  SeqWalk q;
  if (run >= runs) {  // the state after the last token: one thread per sequence and V channels
    if (last == nullptr || run - runs >= d.num_seqs) return;
    q.of(d, (int)(run - runs));
    f32x2 v[P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      load_row<IT, V, W>(d, q, x, state, q.s1 - (W - 1) + j, c, v);
      store_row<V>(last + ((long long)q.n * (W - 1) + j) * d.C + c, v);
    }
    return;
  }
  const long long t0 = run * L, t1 = min(t0 + L, d.total);
  f32x2 wt[W][P], b[P], win[W][P];
  load_taps<V, W>(w, bias, c, wt, b);
  q.find(d, t0);
  for (long long a = t0; a < t1;) {
    const int n = (int)(min(t1, q.s1) - a);  // this run's tokens of the sequence
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<IT, V, W>(d, q, x, state, a - (W - 1) + j, c, win[j + 1]);
    IT* yp = y + a * d.C + c;
    const IT* const src[1] = {x + a * d.ld_x + c};
    const long long ld[1] = {d.ld_x};
    walk_rows<IT, V, 1, kDeep>(src, ld, n, slots + threadIdx.x * (V > 1), [&](int, const f32x2(&in)[1][P]) {
      f32x2 pre[P];
      push<V, W>(win, in[0]);
      taps<V, W>(win, wt, b, pre);
      if (d.silu) silu_row<V>(pre);
      store_row<V>(yp, pre);
      yp += d.C;
    });
    a += n;
    if (a < t1) q.next(d);
  }
}

// dpre of a row from its window and dy: dy silu'(pre), silu'(p) = s + p s (1 - s).
template <int V, int W>
__device__ __forceinline__ void grad_pre(const f32x2 (&win)[W][kPairs<V>], const f32x2 (&wt)[W][kPairs<V>],
                                         const f32x2 (&b)[kPairs<V>], int silu, f32x2 (&g)[kPairs<V>]) {
  if (silu) {
    f32x2 pre[kPairs<V>];
    taps<V, W>(win, wt, b, pre);
    const f32x2 one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
      const f32x2 s = sigmoid2(pre[i]);
      g[i] = mul2(mul2(g[i], s), fma2(pre[i], fma2(s, minus, one), one));
    }
  }
}

// B = 2, T = 4096, C = 6144, bf16, W = 4, from a cold L2: 71 us, 302 MB, 4.3 TB/s (16 warps per SM, 26
// instructions per element).  With four rows in registers 86 us; with a condition on every row's
// window moves besides, so that they are real moves, 120 us.
//
// Blocks of kThreads / cpb runs of L tokens by cpb groups of V channels; a block's sums of dw and
// dbias go to partial[blockIdx.x][W + 1][C].  blockIdx.x >= tiles: dstate, one sequence per run.
template <typename IT, int V, int W>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(ConvDims d, const IT* __restrict__ x,
                                                               const float* __restrict__ w,
                                                               const float* __restrict__ bias,
                                                               const IT* __restrict__ state,
                                                               const IT* __restrict__ dy,
                                                               const IT* __restrict__ dlast, IT* __restrict__ dx,
                                                               IT* __restrict__ dstate, float* __restrict__ partial,
                                                               int L, int cpb, int tiles) {
  constexpr int P = kPairs<V>, kDeep = sizeof(IT) == 2 ? 8 : 4;
  __shared__ Raw<IT, V> slots[V > 1 ? 2 * kDeep * kThreads : 1];
  __shared__ float red[kThreads * V];
  if (d.status && *d.status) return;
  const int subs = kThreads / cpb, sub = threadIdx.x / cpb, cg = threadIdx.x - sub * cpb;
  const long long c = ((long long)blockIdx.y * cpb + cg) * V;
  const bool live = c < d.C;
  SeqWalk q;
  f32x2 wt[W][P], b[P], win[W][P], dwin[W][P];  // win: the last W inputs; dwin: the last W dpre
  f32x2 acc[W + 1][P];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) acc[j][i] = 0;
  if (live) load_taps<V, W>(w, bias, c, wt, b);
  const f32x2 zero[P] = {};

  // windows in front of row u; dpre before it counts as zero
  auto open = [&](long long u) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<IT, V, W>(d, q, x, state, u - (W - 1) + j, c, win[j + 1]);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) dwin[j][i] = 0;
  };
  // dX of row p from the dpre of rows p .. p + W - 1 (dwin[j] = dpre[p + j])
  auto row_grad = [&](long long p, f32x2 (&out)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) out[i] = mul2(wt[W - 1][i], dwin[0][i]);
#pragma unroll
    for (int j = 1; j < W; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) out[i] = fma2(wt[W - 1 - j][i], dwin[j][i], out[i]);
    if (dlast) {
      const long long k = p - (q.s1 - (W - 1));
      if (k >= 0) {
        f32x2 v[P];
        Raw<IT, V> r;
        r.load(dlast + ((long long)q.n * (W - 1) + k) * d.C + c);
        r.get(v);
#pragma unroll
        for (int i = 0; i < P; ++i) out[i] = add2(out[i], v[i]);
      }
    }
  };
  // both windows move on to a row (g: its dy); its dpre is left in dwin[W - 1]
  auto advance = [&](const f32x2(&in)[P], f32x2(&g)[P]) {
    push<V, W>(win, in);
    grad_pre<V, W>(win, wt, b, d.silu, g);
    push<V, W>(dwin, g);
  };

  if ((int)blockIdx.x >= tiles) {
    const long long n = (long long)(blockIdx.x - tiles) * subs + sub;
    if (!live || n >= d.num_seqs) return;
    q.of(d, (int)n);
    open(q.s0);
    for (int k = 0; k < W - 1; ++k) {  // row s0 + k completes the window of row s0 + k - (W - 1)
      const long long u = q.s0 + k;
      if (u < q.s1) {
        Raw<IT, V> rx, rd;
        f32x2 in[P], g[P];
        rx.load(x + u * d.ld_x + c);
        rd.load(dy + u * d.ld_dy + c);
        rx.get(in);
        rd.get(g);
        advance(in, g);
      } else {
        push<V, W>(dwin, zero);
      }
      // state row k is X row s0 - (W - 1) + k: dpre of rows s0 .. s0 + k reach it
      f32x2 out[P];
      row_grad(u - (W - 1), out);
      store_row<V>(dstate + (n * (W - 1) + k) * d.C + c, out);
    }
    return;
  }

  const long long t0 = ((long long)blockIdx.x * subs + sub) * L, t1 = min(t0 + L, d.total);
  if (live && t0 < t1) {
    q.find(d, t0);
    for (long long a = t0; a < t1;) {
      const int n = (int)(min(t1, q.s1) - a);                    // this run's rows of the sequence
      const int stop = (int)min((long long)n + W - 1, q.s1 - a);  // dpre is needed up to here
      open(a);
      IT* op = dx + a * d.C + c;
      auto emit = [&](int u) {  // row u's dpre is in: row u - (W - 1) is complete
        if (u >= W - 1) {
          f32x2 out[P];
          row_grad(a + u - (W - 1), out);
          store_row<V>(op, out);
          op += d.C;
        }
      };
      auto one = [&](int u, const f32x2(&in)[P], f32x2(&g)[P]) {
        advance(in, g);
        if (u < n) {
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) acc[j][i] = fma2(dwin[W - 1][i], win[j][i], acc[j][i]);
#pragma unroll
          for (int i = 0; i < P; ++i) acc[W][i] = add2(acc[W][i], dwin[W - 1][i]);
        }
        emit(u);
      };
      const IT* const src[2] = {x + a * d.ld_x + c, dy + a * d.ld_dy + c};
      const long long ld[2] = {d.ld_x, d.ld_dy};
      walk_rows<IT, V, 2, kDeep>(src, ld, stop, slots + threadIdx.x * (V > 1), [&](int u, f32x2(&in)[2][P]) {
        one(u, in[0], in[1]);
      });
      for (int u = stop; u < n + W - 1; ++u) {  // past the sequence's end: no dpre
        push<V, W>(dwin, zero);
        emit(u);
      }
      a += n;
      if (a < t1) q.next(d);
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) red[(sub * V + i) * cpb + cg] = i & 1 ? hi2(acc[j][i / 2]) : lo2(acc[j][i / 2]);
    __syncthreads();
    for (int k = threadIdx.x; k < cpb * V; k += kThreads) {
      const int i = k / cpb, kg = k - i * cpb;
      float sum = 0.f;
      for (int r = 0; r < subs; ++r) sum += red[(r * V + i) * cpb + kg];
      const long long cc = ((long long)blockIdx.y * cpb + kg) * V + i;
      if (cc < d.C) partial[((long long)blockIdx.x * (W + 1) + j) * d.C + cc] = sum;
    }
  }
}

// V channels of R rows per thread: the taps are read once for them.
template <typename IT, int V, int W, int R>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(int B, int C, long long ld_x, int silu, int num_slots,
                                                             const IT* __restrict__ x, const float* __restrict__ w,
                                                             const float* __restrict__ bias, IT* __restrict__ pool,
                                                             const int32_t* __restrict__ slots,
                                                             IT* __restrict__ y) {
  constexpr int P = kPairs<V>;
  const long long c = ((long long)blockIdx.x * kThreads + threadIdx.x) * V;
  if (c >= C) return;
  const int b0 = blockIdx.y * R;
  Raw<IT, V> r[R][W];
  IT* st[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int b = b0 + i, slot = b < B ? (slots ? slots[b] : b) : -1;
    st[i] = slot >= 0 && slot < num_slots ? pool + (long long)slot * (W - 1) * C + c : nullptr;
    if (st[i]) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) r[i][j].load(st[i] + (long long)j * C);
      r[i][W - 1].load(x + b * ld_x + c);
    }
  }
  f32x2 wt[W][P], bs[P];
  load_taps<V, W>(w, bias, c, wt, bs);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (b0 + i >= B) return;
    f32x2 pre[P] = {};
    if (st[i]) {
      f32x2 win[W][P];
#pragma unroll
      for (int j = 0; j < W; ++j) r[i][j].get(win[j]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) store_row<V>(st[i] + (long long)j * C, win[j + 1]);
      taps<V, W>(win, wt, bs, pre);
      if (silu) silu_row<V>(pre);
    }
    store_row<V>(y + (long long)(b0 + i) * C + c, pre);
  }
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

// Whether every tensor is aligned to kVec elements.
bool quads(std::initializer_list<const void*> ps, size_t el) {
  for (const void* p : ps)
    if (!elem_ok(p, kVec * el)) return false;
  return true;
}

// Launch shape of the backward: channel groups per block and tokens per run.
struct BwdShape {
  int cpb, L;
  long long tiles;
};
BwdShape bwd_shape(const ConvDims& d) {
  BwdShape b;
  const int ncg = (d.C + kVec - 1) / kVec;
  b.cpb = ncg >= 32 ? 32 : ncg >= 16 ? 16 : 8;
  // whole waves of two blocks per SM, as in the forward; runs of 4 to 256 tokens (long runs also keep
  // the partial rows few)
  const long long subs = kThreads / b.cpb, gy = (ncg + b.cpb - 1) / b.cpb;
  const long long per_wave = 2 * kSmCount > gy ? 2 * kSmCount / gy : 1;
  const long long waves = (d.total + per_wave * subs * 256 - 1) / (per_wave * subs * 256), tiles = per_wave * waves;
  const long long L = tiles > 0 ? (d.total + tiles * subs - 1) / (tiles * subs) : 4;
  b.L = (int)(L < 4 ? 4 : L);
  b.tiles = (d.total + b.L * subs - 1) / (b.L * subs);
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
  using VN = std::integral_constant<int, kVec>;
  using V1 = std::integral_constant<int, 1>;
  if (dt == GDR_DTYPE_BF16) return vec ? width(__nv_bfloat16{}, VN{}) : width(__nv_bfloat16{}, V1{});
  return vec ? width(float{}, VN{}) : width(float{}, V1{});
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
  const bool vec = d.C % kVec == 0 && d.ld_x % kVec == 0 && quads({x, y, state, last}, el) && vec_ok(w);
  const long long ncg = vec ? d.C / kVec : d.C;
  // Runs of equal length in whole waves of blocks: as many tokens as one wave needs, at
  // most 128 (a run reads W - 1 rows of its neighbour's again), at least 4.
  const long long wave = (long long)kFwdBlocks * kSmCount * kThreads, per = (d.total * ncg + wave - 1) / wave, waves = (per + 127) / 128;
  long long run = waves > 0 ? (per + waves - 1) / waves : 4;
  run = (run + 3) / 4 * 4;
  const int L = (int)(run < 4 ? 4 : run);
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
  const bool vec = d.C % kVec == 0 && d.ld_x % kVec == 0 && d.ld_dy % kVec == 0 &&
                   quads({x, dy, dx, state, dlast, dstate}, el) && vec_ok(w);
  const BwdShape b = bwd_shape(d);
  const int subs = kThreads / b.cpb;
  const long long gx = b.tiles + (dstate ? ((long long)d.num_seqs + subs - 1) / subs : 0);
  const int ncg = vec ? d.C / kVec : d.C;
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
  const bool vec = d.C % kVec == 0 && d.ld_x % kVec == 0 && quads({x, y, pool}, el) && vec_ok(w);
  const int ncg = vec ? d.C / kVec : d.C, gx = (ncg + kThreads - 1) / kThreads;
  const bool four = (long long)gx * ((p->B + 3) / 4) >= 2 * kSmCount;  // rows enough to keep every SM busy
  const int rows = four ? 4 : 1;
  if ((p->B + rows - 1) / rows > 65535) return GDR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)((p->B + rows - 1) / rows));
  return status_of(by_type(p->dtype, vec, p->W, [&](auto it, auto v, auto wd) {
    using IT = decltype(it);
    constexpr int V = decltype(v)::value, W = decltype(wd)::value;
    const auto kernel = four ? conv_step_kernel<IT, V, W, 4> : conv_step_kernel<IT, V, W, 1>;
    kernel<<<grid, kThreads, 0, s>>>(p->B, d.C, d.ld_x, d.silu, p->num_slots, (const IT*)x, w, bias, (IT*)pool, slots, (IT*)y);
    stage_mark(s, "conv_step");
    return cudaGetLastError();
  }));
}

}  // extern "C"
