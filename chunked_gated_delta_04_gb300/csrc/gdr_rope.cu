// gdr_rope.cu -- rotary positions (include/gdr_attn.h): y_a = scale (x_a cos t - x_b sin t),
// y_b = scale (x_b cos t + x_a sin t), t = +- position * freq, per pair of features of every head.
//
// The angle: a frequency in turns per position is the 64-bit fraction F, so position * F mod 2^64 is the fraction of a
// turn, exact but for F's own rounding (2^-64 turns times the position); its high word goes to sincospi.  In fp32 the
// angle of position 100000 at one radian per position would be off by 4e-3.
// Bound by memory: every feature is read and written once.  A thread keeps the sines of its pairs in registers and takes
// several heads of its token, so that they are worked out once for four heads or more where there are tokens enough.
#include <cmath>

#include "gdr_attn.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;

struct RopeDims {
  long long tokens;
  int T, Hq, Hk, D, R, num_seqs;
  const int32_t* cu;
  int inverse;
  float scale;
  long long ld_q, ld_k;
  int chunks, rot_chunks;  // of a head: rotated ones, then those that are passed on
  int lanes;               // threads that share a token's heads
};

// freq / (2 pi) mod 1 in units of 2^-64: the mantissa times 2^66 / (2 pi), shifted by the exponent.
__device__ __forceinline__ unsigned long long turns_of(double freq) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(freq);
  const int e = (int)(bits >> 52 & 0x7FF) - 1023;
  if (e < -1022) return 0;  // zero (and what is too small to turn anything)
  const unsigned long long m = bits << 11 | 1ull << 63;         // freq = m 2^(e - 63)
  const unsigned long long t = __umul64hi(m, 11743562013128004906ull);  // m 2^66 / (2 pi) / 2^64 = turns 2^(65 - e)
  const int down = 1 - e;
  const unsigned long long f = down >= 64 ? 0 : down >= 0 ? t >> down : -down >= 64 ? 0 : t << -down;
  return bits >> 63 ? 0ull - f : f;
}

// V consecutive elements as fp32.
template <typename IT, int V>
__device__ __forceinline__ void load_v(const IT* p, float (&v)[V]) {
  constexpr int N = 16 / sizeof(IT);
  if constexpr (V < N) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(p[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += N) {
      alignas(16) IT x[N];
      *reinterpret_cast<uint4*>(x) = __ldg(reinterpret_cast<const uint4*>(p + i));
#pragma unroll
      for (int j = 0; j < N; ++j) v[i + j] = to_f32(x[j]);
    }
  }
}
template <typename IT, int V>
__device__ __forceinline__ void put_v(IT* p, const float (&v)[V]) {
  if constexpr (V < (int)(16 / sizeof(IT))) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = from_f32<IT>(v[i]);
  } else {
    store_v<V>(p, v);
  }
}

// V pairs per thread; Pairs: neighbouring features, else halves apart.
template <typename IT, int V, bool Neighbours>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeDims d, const IT* __restrict__ q, const IT* __restrict__ k,
                                                        const double* __restrict__ freqs, const int32_t* __restrict__ positions,
                                                        IT* __restrict__ q_out, IT* __restrict__ k_out, uint32_t* __restrict__ status) {
  if (d.cu) {  // places come from cu_seqlens: every block looks through them, the first reports
    bool bad = false;
    for (int n = threadIdx.x; n < d.num_seqs; n += kThreads) bad |= d.cu[n] > d.cu[n + 1];
    if (threadIdx.x == 0) bad |= d.cu[0] != 0 || d.cu[d.num_seqs] != d.T;
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = bad ? kDevErrBadCuSeqlens : 0u;
    if (bad) return;
  }
  const long long x = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int c = (int)(x % d.chunks), lane = (int)(x / d.chunks % d.lanes);
  const long long token = x / ((long long)d.chunks * d.lanes);
  if (token >= d.tokens) return;
  const int heads = d.Hq + d.Hk;
  const IT *qt = q + token * d.ld_q, *kt = k + token * d.ld_k;
  IT *qo = q_out + token * d.Hq * d.D, *ko = k_out + token * d.Hk * d.D;
  if (c >= d.rot_chunks) {  // passed on as it is
    constexpr int N = V * 2;
    const int at = d.R + (c - d.rot_chunks) * N, n = min(N, d.D - at);
    for (int h = lane; h < heads; h += d.lanes) {
      const IT* from = h < d.Hq ? qt + h * d.D : kt + (h - d.Hq) * d.D;
      IT* to = h < d.Hq ? qo + h * d.D : ko + (h - d.Hq) * d.D;
      if constexpr (V == 1) {
        for (int i = 0; i < n; ++i) to[at + i] = from[at + i];
      } else {  // whole 16 bytes: V divides what is left
#pragma unroll
        for (int i = 0; i < N; i += 16 / sizeof(IT))
          if (i < n) *reinterpret_cast<uint4*>(to + at + i) = __ldg(reinterpret_cast<const uint4*>(from + at + i));
      }
    }
    return;
  }
  const long long pos = positions ? (long long)positions[token]
                        : d.cu    ? token - d.cu[seq_of(d.cu, d.num_seqs, token)]
                                  : token % d.T;
  float cs[V], sn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    unsigned long long a = (unsigned long long)pos * turns_of(freqs[c * V + i]);
    if (d.inverse) a = 0ull - a;
    sincospif((float)(int)(a >> 32) * 0x1p-31f, &sn[i], &cs[i]);
    sn[i] *= d.scale;
    cs[i] *= d.scale;
  }
  const int pa = Neighbours ? 2 * V * c : V * c, pb = Neighbours ? 0 : d.R / 2 + V * c;
#pragma unroll 2
  for (int h = lane; h < heads; h += d.lanes) {
    const IT* from = h < d.Hq ? qt + h * d.D : kt + (h - d.Hq) * d.D;
    IT* to = h < d.Hq ? qo + h * d.D : ko + (h - d.Hq) * d.D;
    if constexpr (Neighbours) {
      float v[2 * V];
      load_v<IT, 2 * V>(from + pa, v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = fmaf(a, cs[i], -b * sn[i]);
        v[2 * i + 1] = fmaf(b, cs[i], a * sn[i]);
      }
      put_v<IT, 2 * V>(to + pa, v);
    } else {
      float va[V], vb[V], ya[V], yb[V];
      load_v<IT, V>(from + pa, va);
      load_v<IT, V>(from + pb, vb);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ya[i] = fmaf(va[i], cs[i], -vb[i] * sn[i]);
        yb[i] = fmaf(vb[i], cs[i], va[i] * sn[i]);
      }
      put_v<IT, V>(to + pa, ya);
      put_v<IT, V>(to + pb, yb);
    }
  }
}

gdr_status resolve_rope(const gdr_rope_problem* p, RopeDims* d) {
  if (p == nullptr || p->B < 0 || p->T < 0 || p->Hq <= 0 || p->Hk < 0 || p->num_seqs < 0) return GDR_ERR_INVALID_ARG;
  if (p->D <= 0 || p->R <= 0 || p->R % 2 != 0 || p->R > p->D || !dtype_ok(p->dtype)) return GDR_ERR_INVALID_ARG;
  if ((p->interleaved != 0 && p->interleaved != 1) || (p->inverse != 0 && p->inverse != 1) || !std::isfinite(p->scale)) return GDR_ERR_INVALID_ARG;
  const long long wq = (long long)p->Hq * p->D, wk = (long long)p->Hk * p->D;
  if ((p->ld_q && p->ld_q < wq) || (p->ld_k && p->ld_k < wk) || p->ld_q < 0 || p->ld_k < 0) return GDR_ERR_INVALID_ARG;
  if (p->cu_seqlens ? p->B != 1 || p->num_seqs < 1 : p->num_seqs != p->B) return GDR_ERR_INVALID_ARG;
  if (p->D > 1024 || (long long)p->Hq + p->Hk > 65536) return GDR_ERR_UNSUPPORTED;
  d->tokens = (long long)p->B * p->T;
  if (d->tokens >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  d->T = p->T, d->Hq = p->Hq, d->Hk = p->Hk, d->D = p->D, d->R = p->R, d->num_seqs = p->num_seqs;
  d->cu = p->cu_seqlens;
  d->inverse = p->inverse;
  d->scale = p->scale;
  d->ld_q = p->ld_q ? p->ld_q : wq, d->ld_k = p->ld_k ? p->ld_k : wk;
  return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_rope_workspace_bytes(const gdr_rope_problem* p) {
  RopeDims d;
  return resolve_rope(p, &d) == GDR_OK && d.cu ? 256 : 0;
}

gdr_status gdr_rope(const gdr_rope_problem* p, const void* q, const void* k, const double* freqs, const int32_t* positions,
                    void* q_out, void* k_out, void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  RopeDims d;
  const gdr_status st = resolve_rope(p, &d);
  if (st != GDR_OK) return st;
  if (!freqs || (d.tokens > 0 && (!q || !q_out || (d.Hk > 0 && (!k || !k_out))))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(q, el) || !elem_ok(k, el) || !elem_ok(q_out, el) || !elem_ok(k_out, el) || !elem_ok(freqs, 8) || !elem_ok(positions, 4) ||
      !elem_ok(d.cu, 4) || ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  if (positions) d.cu = nullptr;
  if (d.cu && (!workspace || workspace_bytes < 256)) return GDR_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  // 16 bytes at a time: 8 (bf16) or 4 (fp32) pairs halves apart, half as many neighbouring ones
  const int n16 = (int)(16 / el), V = p->interleaved ? n16 / 2 : n16;
  const bool vec = vec_ok(q) && vec_ok(k) && vec_ok(q_out) && vec_ok(k_out) && d.ld_q % n16 == 0 && d.ld_k % n16 == 0 && d.D % n16 == 0 &&
                   d.R / 2 % V == 0 && d.R % n16 == 0;
  const int v = vec ? V : 1;
  d.rot_chunks = d.R / 2 / v;
  d.chunks = d.rot_chunks + (d.D - d.R + 2 * v - 1) / (2 * v);
  // Heads per thread: eight, so that a sine serves eight times; fewer while that leaves SMs without threads (2048 each).
  const int heads = d.Hq + d.Hk;
  int per = 8;
  while (per > 1 && d.tokens * d.chunks * ((heads + per - 1) / per) < 2048ll * kSmCount) per /= 2;
  d.lanes = (heads + per - 1) / per;
  const long long grid = d.tokens == 0 ? (d.cu ? 1 : 0) : (d.tokens * d.chunks * d.lanes + kThreads - 1) / kThreads;
  if (grid == 0) return GDR_OK;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  auto go = [&](auto it, auto vv, auto nb) {
    using IT = decltype(it);
    rope_kernel<IT, decltype(vv)::value, decltype(nb)::value><<<(unsigned)grid, kThreads, 0, s>>>(
        d, (const IT*)q, (const IT*)k, freqs, positions, (IT*)q_out, (IT*)k_out, (uint32_t*)workspace);
    stage_mark(s, "rope");
    return cudaGetLastError();
  };
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C4 = std::integral_constant<int, 4>;
  using C8 = std::integral_constant<int, 8>;
  const std::true_type nb{};
  const std::false_type halves{};
  if (p->dtype == GDR_DTYPE_BF16) {
    const __nv_bfloat16 t{};
    if (p->interleaved) return status_of(vec ? go(t, C4{}, nb) : go(t, C1{}, nb));
    return status_of(vec ? go(t, C8{}, halves) : go(t, C1{}, halves));
  }
  if (p->interleaved) return status_of(vec ? go(0.f, C2{}, nb) : go(0.f, C1{}, nb));
  return status_of(vec ? go(0.f, C4{}, halves) : go(0.f, C1{}, halves));
}

}  // extern "C"
