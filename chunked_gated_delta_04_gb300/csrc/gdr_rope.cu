// gdr_rope.cu -- rotary positions (include/gdr_attn.h): y_a = scale (x_a cos t - x_b sin t),
// y_b = scale (x_b cos t + x_a sin t), t = +- position * freq, per pair of features of every head.
//
// The angle: a frequency in turns per position is the 64-bit fraction F, so position * F mod 2^64 is the fraction of a
// turn, exact but for F's own rounding (2^-64 turns times the position); its high word goes to sincospi.  In fp32 the
// angle of position 100000 at one radian per position would be off by 4e-3.
// Bound by memory: every feature is read and written once.  A thread keeps the sines of its pairs in registers and takes
// several heads of its token, so that they are worked out once for up to eight; the first two heads' loads are under way
// meanwhile.  Features that are passed on have warps of their own.  B = 2, T = 4096, 16 + 16 heads of 128, 64 features turned, bf16, forward
// and backward: 51 us, 5.3 TB/s (66 us with the loads behind the sines; 73 us with both kinds of threads in one warp and four heads' loads;
// 57 and 65 us with the next one or two heads' loads in front of a head's stores, whose registers cost warps).  Element by element, where base
// or strides are off 16 bytes, one way takes 53 us for 25, in fp32 67 for 45.
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
  int rot_chunks, pass_chunks;  // of a head: threads that rotate, threads that pass features on
  int lanes;                    // threads that share a token's heads
  long long rotating;           // threads that rotate, of all tokens; the others' warps come behind them
  int narrow;                   // both kinds' places fit 32 bits: 64-bit divisions cost as much as the rotation
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

// V consecutive elements, as they are stored: 16-byte pieces, or one element.
template <typename IT, int V>
struct Raw {
  static constexpr int N = 16 / (int)sizeof(IT);
  alignas(V >= N ? 16 : sizeof(IT)) IT x[V];
  __device__ __forceinline__ void load(const IT* p) {
    if constexpr (V >= N) {
#pragma unroll
      for (int i = 0; i < V; i += N) *reinterpret_cast<uint4*>(x + i) = *reinterpret_cast<const uint4*>(p + i);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = p[i];
    }
  }
};
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
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeDims d, const IT* q, const IT* k,
                                                        const double* freqs, const int32_t* positions,
                                                        IT* q_out, IT* k_out, uint32_t* status) {
  launch_wait();
  launch_next();
  if (d.cu) {  // places come from cu_seqlens: every block looks through them, the first reports
    bool bad = false;
    for (int n = threadIdx.x; n < d.num_seqs; n += kThreads) bad |= d.cu[n] > d.cu[n + 1];
    if (threadIdx.x == 0) bad |= d.cu[0] != 0 || d.cu[d.num_seqs] != d.T;
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = bad ? kDevErrBadCuSeqlens : 0u;
    if (bad) return;
  }
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const bool rotates = at < d.rotating;
  const long long x = rotates ? at : at - d.rotating;
  const int chunks = rotates ? d.rot_chunks : d.pass_chunks;
  int c, lane;
  long long token;
  if (d.narrow) {
    const uint32_t y = (uint32_t)x / (uint32_t)max(chunks, 1);
    c = (int)((uint32_t)x - y * (uint32_t)chunks);
    token = y / (uint32_t)d.lanes;
    lane = (int)(y - (uint32_t)token * (uint32_t)d.lanes);
  } else {
    const long long y = x / max(chunks, 1);
    c = (int)(x - y * chunks);
    token = y / d.lanes;
    lane = (int)(y - token * d.lanes);
  }
  if (token >= d.tokens) return;
  const int heads = d.Hq + d.Hk;
  const IT *qt = q + token * d.ld_q, *kt = k + token * d.ld_k;
  IT *qo = q_out + token * d.Hq * d.D, *ko = k_out + token * d.Hk * d.D;
  if (!rotates) {  // passed on as it is
    if (chunks == 0) return;
    constexpr int N = V * 2;
    const int at = d.R + c * N, n = min(N, d.D - at);
#pragma unroll 4
    for (int h = lane; h < heads; h += d.lanes) {
      const IT* from = h < d.Hq ? qt + h * d.D : kt + (h - d.Hq) * d.D;
      IT* to = h < d.Hq ? qo + h * d.D : ko + (h - d.Hq) * d.D;
      if constexpr (V == 1) {
        for (int i = 0; i < n; ++i) to[at + i] = from[at + i];
      } else {  // whole 16 bytes: V divides what is left
#pragma unroll
        for (int i = 0; i < N; i += 16 / sizeof(IT))
          if (i < n) *reinterpret_cast<uint4*>(to + at + i) = *reinterpret_cast<const uint4*>(from + at + i);
      }
    }
    return;
  }
  constexpr int H = 2;  // heads whose loads are under way together
  const int pa = Neighbours ? 2 * V * c : V * c, pb = d.R / 2 + V * c;
  Raw<IT, Neighbours ? 2 * V : V> xa[H];
  Raw<IT, Neighbours ? 1 : V> xb[H];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int h = h0 + i * d.lanes;
      if (h >= heads) break;
      const IT* from = h < d.Hq ? qt + h * d.D : kt + (h - d.Hq) * d.D;
      xa[i].load(from + pa);
      if constexpr (!Neighbours) xb[i].load(from + pb);
    }
  };
  load(lane);
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
  for (int h0 = lane; h0 < heads; h0 += H * d.lanes) {
    if (h0 != lane) load(h0);
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const int h = h0 + k * d.lanes;
      if (h >= heads) break;
      IT* to = h < d.Hq ? qo + h * d.D : ko + (h - d.Hq) * d.D;
      if constexpr (Neighbours) {
        float v[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float a = to_f32(xa[k].x[2 * i]), b = to_f32(xa[k].x[2 * i + 1]);
          v[2 * i] = fmaf(a, cs[i], -b * sn[i]);
          v[2 * i + 1] = fmaf(b, cs[i], a * sn[i]);
        }
        put_v<IT, 2 * V>(to + pa, v);
      } else {
        float ya[V], yb[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float a = to_f32(xa[k].x[i]), b = to_f32(xb[k].x[i]);
          ya[i] = fmaf(a, cs[i], -b * sn[i]);
          yb[i] = fmaf(b, cs[i], a * sn[i]);
        }
        put_v<IT, V>(to + pa, ya);
        put_v<IT, V>(to + pb, yb);
      }
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
  d.pass_chunks = (d.D - d.R + 2 * v - 1) / (2 * v);
  const int chunks = d.rot_chunks + d.pass_chunks;
  // Heads per thread: eight, so that a sine serves eight times; fewer while that leaves SMs without threads (2048 each).
  const int heads = d.Hq + d.Hk;
  int per = 8;
  while (per > 1 && d.tokens * chunks * ((heads + per - 1) / per) < 2048ll * kSmCount) per /= 2;
  d.lanes = (heads + per - 1) / per;
  d.rotating = d.tokens * d.lanes * d.rot_chunks;
  // the last block's threads behind the last place count, too
  d.narrow = d.tokens * d.lanes * (d.rot_chunks > d.pass_chunks ? d.rot_chunks : d.pass_chunks) + kThreads < 1ll << 32;
  const long long grid = d.tokens == 0 ? (d.cu ? 1 : 0) : (d.tokens * chunks * d.lanes + kThreads - 1) / kThreads;
  if (grid == 0) return GDR_OK;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  auto go = [&](auto it, auto vv, auto nb) {
    using IT = decltype(it);
    const cudaError_t e = attn_launch(rope_kernel<IT, decltype(vv)::value, decltype(nb)::value>, grid, kThreads, 0, 1, s, d, (const IT*)q,
                                      (const IT*)k, freqs, positions, (IT*)q_out, (IT*)k_out, (uint32_t*)workspace);
    if (e != cudaSuccess) return e;
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
