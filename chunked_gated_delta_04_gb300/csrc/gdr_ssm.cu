// gdr_ssm.cu -- the selective state space scan, forward and single token (include/gdr_block.h):
//
//   D_t = softplus(dt_t + dt_bias),  h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,  y_t = sum_n C_t h_t + Dskip x_t
//
// Every (channel, state) pair decays at a rate of its own, so there is no matrix product whose
// factors stay in range: the recurrence runs token by token in fp32 registers.  NL = N / 4 lanes
// share a channel, four states each; the sum over n runs over those lanes for four tokens at a
// time.  A block holds CB channels; it stages 16 tokens of D_t, D_t x_t, B_t and C_t in shared memory (formed once
// per token and channel) while the loads of the next 16 are in flight.  Bound by arithmetic from
// N = 16 on: per (token, channel, state) one exponential and four multiply-adds, against
// 6 / N bytes in bf16.
//
// Where the channels do not fill the GPU the sequence is cut into segments: a first pass finds
// every segment's end state from zero, a scan joins them (the decay over a segment is exp(A sum D_t),
// one exponential), and the full pass runs all segments side by side from their true states.
#include "gdr_ssm.cuh"

namespace gdr {
namespace {

constexpr int fwd_threads(int NL) { return NL <= 4 ? 128 : 32 * NL; }

enum SsmMode { kFull, kEndState, kStartGrad };

// kFull: y (and states, S_T).  kEndState: R[u] = end state of unit u from zero, and sum of D_t.
// kStartGrad (in reverse): R[u] = gradient of the state in front of unit u from a zero gradient
// behind it; x is dy, and C plays B's part.
template <typename IT, int NL, int MODE>
__global__ void __launch_bounds__(fwd_threads(NL))
    ssm_scan_kernel(SsmDims d, const IT* __restrict__ x, long long ld_x, const IT* __restrict__ dt,
                    const float* __restrict__ A, const IT* __restrict__ Bm, long long ld_b,
                    const IT* __restrict__ Cm, const float* __restrict__ Dskip, const float* __restrict__ dt_bias,
                    const float* __restrict__ start, int start_per_unit, IT* __restrict__ y, float* __restrict__ S_T,
                    float* __restrict__ h_saved, float* __restrict__ R, float* __restrict__ sum_delta) {
  constexpr int NT = fwd_threads(NL), CB = NT / NL, N = 4 * NL;
  constexpr int PER = kTile * CB / NT, PB = (kTile * N + NT - 1) / NT;
  __shared__ float sd[kTile][CB], su[kTile][CB], sx[MODE == kFull ? kTile : 1][CB];
  __shared__ __align__(16) float sB[kTile][N], sC[MODE == kFull ? kTile : 1][N];
  if (ssm_bad(d)) return;
  const int tid = threadIdx.x, ln = tid % NL, ch = tid / NL;
  const int blocks = (d.Dg + CB - 1) / CB, grp = blockIdx.x / blocks, c0 = (blockIdx.x - grp * blocks) * CB;
  const int nch = min(CB, d.Dg - c0);           // live channels of this block
  const long long dc0 = (long long)grp * d.Dg + c0;  // its first channel
  const bool live = ch < nch;
  const long long dch = dc0 + ch;
  float A2[4] = {};
  if (live) {
    const float4 a = *reinterpret_cast<const float4*>(A + dch * N + 4 * ln);
    // finite, so that D = 0 past the end gives exp(0) = 1 also for A = -infinity
    A2[0] = fmaxf(a.x * kLog2e, -kBig); A2[1] = fmaxf(a.y * kLog2e, -kBig);
    A2[2] = fmaxf(a.z * kLog2e, -kBig); A2[3] = fmaxf(a.w * kLog2e, -kBig);
  }
  const float skip = MODE == kFull && Dskip && live ? Dskip[dch] : 0.f;

  const long long units = ssm_unit_count(d);
  for (long long un = blockIdx.y; un < units; un += gridDim.y) {
    const SsmUnit q = ssm_unit(d, un);
    float h[4] = {};
    if (MODE == kFull && start && live) {
      const long long at = start_per_unit ? un : q.seq;
      const float4 v = *reinterpret_cast<const float4*>(start + (at * d.D + dch) * N + 4 * ln);
      h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
    }
    float dsum = 0.f;
    const int tiles = (q.len + kTile - 1) / kTile;
    IT px[PER], pd[PER], pB[PB], pC[PB];
    auto fetch = [&](int tile) {
      const int base = (MODE == kStartGrad ? tiles - 1 - tile : tile) * kTile;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * NT + tid, t = base + e / CB, c = e % CB;
        const bool in = t < q.len && c < nch;
        px[i] = in ? x[(long long)(q.t0 + t) * ld_x + dc0 + c] : from_f32<IT>(0.f);
        pd[i] = in ? dt[(long long)(q.t0 + t) * d.ld_dt + dc0 + c] : from_f32<IT>(0.f);
      }
#pragma unroll
      for (int i = 0; i < PB; ++i) {
        const int e = i * NT + tid, t = base + e / N, n = e % N;
        const bool in = e < kTile * N && t < q.len;
        pB[i] = in ? Bm[(long long)(q.t0 + t) * ld_b + grp * N + n] : from_f32<IT>(0.f);
        if (MODE == kFull) pC[i] = in ? Cm[(long long)(q.t0 + t) * d.ld_c + grp * N + n] : from_f32<IT>(0.f);
      }
    };
    if (tiles > 0) fetch(0);
    for (int tile = 0; tile < tiles; ++tile) {
      const int base = (MODE == kStartGrad ? tiles - 1 - tile : tile) * kTile;
      __syncthreads();  // the previous tile's readers are done
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * NT + tid, t = e / CB, c = e % CB;
        const bool in = base + t < q.len && c < nch;
        const float xv = to_f32(px[i]);
        float raw = to_f32(pd[i]);
        if (in && dt_bias) raw += dt_bias[dc0 + c];
        float dl = 0.f;  // past the end: D = 0 leaves the state as it is
        if (in) dl = d.softplus ? softplus_f(raw, nullptr) : raw;
        sd[t][c] = dl;
        su[t][c] = MODE == kStartGrad ? xv : dl * xv;
        if (MODE == kFull) sx[t][c] = xv;
      }
#pragma unroll
      for (int i = 0; i < PB; ++i) {
        const int e = i * NT + tid;
        if (e < kTile * N) {
          sB[e / N][e % N] = to_f32(pB[i]);
          if (MODE == kFull) sC[e / N][e % N] = to_f32(pC[i]);
        }
      }
      __syncthreads();
      if (tile + 1 < tiles) fetch(tile + 1);
      if (MODE == kFull && h_saved && live)
        *reinterpret_cast<float4*>(h_saved + ((q.tile0 + tile) * d.D + dch) * N + 4 * ln) =
            make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
      for (int t4 = 0; t4 < kTile; t4 += 4) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = MODE == kStartGrad ? kTile - 1 - (t4 + i) : t4 + i;
          const float dl = sd[t][ch], uu = su[t][ch];
          const float4 b = *reinterpret_cast<const float4*>(&sB[t][4 * ln]);
          const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = ex2f(dl * A2[j]);
            h[j] = MODE == kStartGrad ? a * fmaf(uu, bb[j], h[j]) : fmaf(a, h[j], uu * bb[j]);
          }
          if (MODE == kFull) {
            const float4 c = *reinterpret_cast<const float4*>(&sC[t][4 * ln]);
            p[i] = fmaf(h[0], c.x, fmaf(h[1], c.y, fmaf(h[2], c.z, h[3] * c.w)));
          } else {
            dsum += dl;
          }
        }
        if (MODE == kFull) {
          LaneSum<NL>::run(p, ln);
          if (LaneSum<NL>::holds(ln)) {
#pragma unroll
            for (int k = 0; k < LaneSum<NL>::kKeep; ++k) {
              const int t = t4 + LaneSum<NL>::tok(ln) + k;
              su[t][ch] = fmaf(skip, sx[t][ch], p[k]);  // D_t x_t of these tokens has been used
            }
          }
        }
      }
      if (MODE == kFull) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = i * NT + tid, t = e / CB, c = e % CB;
          if (base + t < q.len && c < nch) y[(long long)(q.t0 + base + t) * d.D + dc0 + c] = from_f32<IT>(su[t][c]);
        }
      }
    }
    if (live) {
      const float4 v = make_float4(h[0], h[1], h[2], h[3]);
      if (MODE == kFull) {
        if (S_T && q.last) *reinterpret_cast<float4*>(S_T + ((long long)q.seq * d.D + dch) * N + 4 * ln) = v;
      } else {
        *reinterpret_cast<float4*>(R + (un * d.D + dch) * N + 4 * ln) = v;
        if (ln == 0) sum_delta[un * d.D + dch] = dsum;
      }
    }
  }
}

// Joins the segments of every sequence: cur = edge; in order (backward: reversed) of its units,
// R[u] <- cur, cur <- exp(A sum D) cur + R[u].  One thread per (sequence, channel, state); the
// loads of the next four units are in flight while four are joined.
__global__ void __launch_bounds__(256) ssm_join_kernel(SsmDims d, const float* __restrict__ A,
                                                       const float* __restrict__ edge, float* R,
                                                       const float* __restrict__ sum_delta, int backward) {
  if (ssm_bad(d)) return;
  const long long DN = (long long)d.D * d.N, id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long seq = id / DN, dn = id - seq * DN;
  if (seq >= d.num_seqs) return;
  const long long u0 = d.cu ? d.unit_off[seq] : seq * d.seq_units;
  const int count = d.cu ? d.unit_off[seq + 1] - (int)u0 : d.seq_units;
  const float a2 = fmaxf(A[dn] * kLog2e, -kBig);
  const long long ch = dn / d.N;
  float cur = edge ? edge[seq * DN + dn] : 0.f;
  for (int k = 0; k < count; k += 4) {
    float r[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long u = u0 + (backward ? count - 1 - (k + i) : k + i);
      r[i] = k + i < count ? R[u * DN + dn] : 0.f;
      s[i] = k + i < count ? sum_delta[u * d.D + ch] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long u = u0 + (backward ? count - 1 - (k + i) : k + i);
      if (k + i < count) {
        R[u * DN + dn] = cur;
        cur = fmaf(ex2f(a2 * s[i]), cur, r[i]);
      }
    }
  }
}

// Units and tiles of a packed batch, after the check of cu_seqlens.
__global__ void __launch_bounds__(1024) ssm_index_kernel(const int32_t* __restrict__ cu, int num_seqs, int T, int Lseg,
                                                         uint32_t* __restrict__ status, int* __restrict__ unit_off,
                                                         int* __restrict__ tile_off, int4* __restrict__ units) {
  __shared__ int wu[32], wt[32], s_bad, cu_u, cu_t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_bad = cu[0] != 0 || cu[num_seqs] != T;
    cu_u = cu_t = 0;
  }
  __syncthreads();
  for (int n = tid; n < num_seqs; n += 1024)
    if (cu[n] > cu[n + 1]) s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      status[0] = kDevErrBadCuSeqlens;
      status[1] = 0;
    }
    return;
  }
  for (int base = 0; base < num_seqs; base += 1024) {
    const int n = base + tid;
    int nu = 0, nt = 0;
    if (n < num_seqs) {
      const int L = cu[n + 1] - cu[n];
      nt = L / kTile + (L % kTile != 0);
      nu = max(1, L / Lseg + (L % Lseg != 0));
    }
    int u = nu, t = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int yu = __shfl_up_sync(0xffffffffu, u, o), yt = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) {
        u += yu;
        t += yt;
      }
    }
    if (lane == 31) {
      wu[warp] = u;
      wt[warp] = t;
    }
    __syncthreads();
    int pu = cu_u, pt = cu_t;
    for (int w = 0; w < warp; ++w) {
      pu += wu[w];
      pt += wt[w];
    }
    if (n < num_seqs) {
      unit_off[n] = pu + u - nu;
      tile_off[n] = pt + t - nt;
    }
    __syncthreads();
    if (tid == 1023) {
      cu_u = pu + u;
      cu_t = pt + t;
    }
    __syncthreads();
  }
  const int total = cu_u;
  if (tid == 0) {
    unit_off[num_seqs] = total;
    status[0] = 0;
    status[1] = (uint32_t)total;
  }
  __syncthreads();  // unit_off, tile_off written by this block are read by it below
  for (int u = tid; u < total; u += 1024) {
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (unit_off[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int s = u - unit_off[lo], L = cu[lo + 1] - cu[lo], off = s * Lseg;
    const bool last = L - off <= Lseg;
    units[u] = make_int4((int)((uint32_t)lo | (s == 0 ? 1u << 30 : 0u) | (last ? 1u << 31 : 0u)), cu[lo] + off,
                         min(Lseg, L - off), tile_off[lo] + off / kTile);
  }
}

template <typename IT, int NL>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmDims d, int B, int num_slots, const IT* __restrict__ x,
                                                       const IT* __restrict__ dt, const float* __restrict__ A,
                                                       const IT* __restrict__ Bm, const IT* __restrict__ Cm,
                                                       const float* __restrict__ Dskip,
                                                       const float* __restrict__ dt_bias, float* __restrict__ pool,
                                                       const int32_t* __restrict__ slots, IT* __restrict__ y) {
  constexpr int N = 4 * NL;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const int ln = (int)(id % NL);
  const long long row = id / NL, b = row / d.D;
  const int ch = (int)(row - b * d.D);
  float p = 0.f;
  const bool in = b < B;
  const int slot = in ? (slots ? slots[b] : (int)b) : -1;
  const bool live = slot >= 0 && slot < num_slots;
  float xv = 0.f;
  if (live) {
    const int g = ch / d.Dg;
    float4* hp = reinterpret_cast<float4*>(pool + ((long long)slot * d.D + ch) * N + 4 * ln);
    float4 h = __ldcs(hp);
    const float4 a = *reinterpret_cast<const float4*>(A + (long long)ch * N + 4 * ln);
    xv = to_f32(x[b * d.ld_x + ch]);
    float dl = to_f32(dt[b * d.ld_dt + ch]) + (dt_bias ? dt_bias[ch] : 0.f);
    if (d.softplus) dl = softplus_f(dl, nullptr);
    const IT* bp = Bm + b * d.ld_b + g * N + 4 * ln;
    const IT* cp = Cm + b * d.ld_c + g * N + 4 * ln;
    const float u = dl * xv, d2 = dl * kLog2e;
    h.x = fmaf(ex2f(d2 * fmaxf(a.x, -kBig)), h.x, u * to_f32(bp[0]));
    h.y = fmaf(ex2f(d2 * fmaxf(a.y, -kBig)), h.y, u * to_f32(bp[1]));
    h.z = fmaf(ex2f(d2 * fmaxf(a.z, -kBig)), h.z, u * to_f32(bp[2]));
    h.w = fmaf(ex2f(d2 * fmaxf(a.w, -kBig)), h.w, u * to_f32(bp[3]));
    __stcs(hp, h);
    p = fmaf(h.x, to_f32(cp[0]), fmaf(h.y, to_f32(cp[1]), fmaf(h.z, to_f32(cp[2]), h.w * to_f32(cp[3]))));
  }
#pragma unroll
  for (int o = 1; o < NL; o <<= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
  if (in && ln == 0) y[b * d.D + ch] = from_f32<IT>(live ? fmaf(Dskip ? Dskip[ch] : 0.f, xv, p) : 0.f);
}

int fwd_blocks(const SsmDims& d) {
  const int NL = d.N / 4, CB = fwd_threads(NL) / NL;
  return d.G * ((d.Dg + CB - 1) / CB);
}

template <typename F>
cudaError_t ssm_type(gdr_dtype dt, F f) {
  return dt == GDR_DTYPE_BF16 ? f(__nv_bfloat16{}) : f(float{});
}

unsigned unit_rows(const SsmDims& d) { return (unsigned)(d.max_units < 32768 ? d.max_units : 32768); }

}  // namespace

bool ssm_split(const SsmDims& d) { return d.Lseg < d.T; }

gdr_status resolve_ssm(const gdr_ssm_problem* p, bool step, SsmDims* d) {
  if (p == nullptr || p->B < 0 || p->T < 0 || p->D <= 0 || p->N <= 0 || p->G <= 0 || p->num_seqs < 0)
    return GDR_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || p->D % p->G != 0 || (p->dt_softplus != 0 && p->dt_softplus != 1)) return GDR_ERR_INVALID_ARG;
  const long long gn = (long long)p->G * p->N;
  if ((p->ld_x && p->ld_x < p->D) || (p->ld_dt && p->ld_dt < p->D) || (p->ld_dy && p->ld_dy < p->D) ||
      (p->ld_b && p->ld_b < gn) || (p->ld_c && p->ld_c < gn))
    return GDR_ERR_INVALID_ARG;
  if (step) {
    if (p->T != 1 || p->cu_seqlens || p->num_slots < 0) return GDR_ERR_INVALID_ARG;
  } else if (p->cu_seqlens ? p->B != 1 || p->num_seqs < 1 : p->num_seqs != p->B) {
    return GDR_ERR_INVALID_ARG;
  }
  if (p->N != 4 && p->N != 8 && p->N != 16 && p->N != 32 && p->N != 64) return GDR_ERR_UNSUPPORTED;
  if (p->D > (1 << 24) || (long long)p->B * p->T >= (1ll << 30) || p->num_seqs >= (1 << 30) || gn >= (1ll << 31))
    return GDR_ERR_UNSUPPORTED;
  *d = SsmDims{};
  d->D = p->D;
  d->N = p->N;
  d->G = p->G;
  d->Dg = p->D / p->G;
  d->T = p->T;
  d->num_seqs = p->num_seqs;
  d->softplus = p->dt_softplus;
  d->total = (long long)p->B * p->T;
  d->ld_x = p->ld_x ? p->ld_x : p->D;
  d->ld_dt = p->ld_dt ? p->ld_dt : p->D;
  d->ld_dy = p->ld_dy ? p->ld_dy : p->D;
  d->ld_b = p->ld_b ? p->ld_b : gn;
  d->ld_c = p->ld_c ? p->ld_c : gn;
  d->cu = p->cu_seqlens;
  // One segment per sequence where the channels alone give every SM about two blocks; else segments
  // of at least 64 tokens, enough of them for four blocks per SM.
  const long long blocks = fwd_blocks(*d), whole = (d->T + kTile - 1) / kTile * (long long)kTile;
  d->Lseg = (int)(whole < kTile ? kTile : whole);
  if (!step && blocks * d->num_seqs < 2 * kSmCount) {
    const long long want = (4ll * kSmCount + blocks - 1) / blocks;  // segments over all sequences
    long long L = (d->total / want + kTile - 1) / kTile * kTile;
    if (L < 64) L = 64;
    if (L < d->Lseg) d->Lseg = (int)L;
  }
  const long long su = d->T == 0 ? 1 : (d->T + (long long)d->Lseg - 1) / d->Lseg;
  const long long stl = (d->T + (long long)kTile - 1) / kTile;
  d->seq_units = (int)su;
  d->seq_tiles = (int)stl;
  d->max_units = d->cu ? (long long)d->T / d->Lseg + d->num_seqs : d->num_seqs * su;
  d->max_tiles = d->cu ? (long long)d->T / kTile + d->num_seqs : d->num_seqs * stl;
  return GDR_OK;
}

SsmWorkspace ssm_workspace(const SsmDims& d, char* base, bool backward) {
  SsmWorkspace w = {};
  size_t off = 0;
  auto take = [&](size_t bytes) -> char* {
    char* p = base ? base + off : nullptr;
    off += block_align(bytes);
    return p;
  };
  w.status = (uint32_t*)take(256);
  if (d.cu) {
    w.unit_off = (int*)take(sizeof(int) * 2 * ((size_t)d.num_seqs + 1));  // unit offsets, then tile offsets
    w.units = (int4*)take(sizeof(int4) * (size_t)d.max_units);
  }
  if (ssm_split(d)) {
    w.R = (float*)take(sizeof(float) * (size_t)d.max_units * d.D * d.N);
    w.sum_delta = (float*)take(sizeof(float) * (size_t)d.max_units * d.D);
  }
  if (backward) {
    const int cb = ssm_bwd_channels(d.N);
    w.grads = (float*)take(sizeof(float) * (size_t)ssm_bwd_rows(d) * (d.N + 2) * d.D);
    w.bc = (float*)take(sizeof(float) * (size_t)((d.Dg + cb - 1) / cb) * d.total * d.G * 2 * d.N);
  }
  w.bytes = off;
  return w;
}

cudaError_t ssm_launch_index(SsmDims* d, const SsmWorkspace& w, cudaStream_t s) {
  if (!d->cu) return cudaSuccess;
  d->status = w.status;
  d->unit_off = w.unit_off;
  d->units = w.units;
  ssm_index_kernel<<<1, 1024, 0, s>>>(d->cu, d->num_seqs, d->T, d->Lseg, w.status, w.unit_off,
                                      w.unit_off + d->num_seqs + 1, w.units);
  stage_mark(s, "ssm_index");
  return cudaGetLastError();
}

cudaError_t ssm_launch_boundaries(const SsmDims& d, gdr_dtype dt, const SsmInputs& in, const float* edge,
                                  const SsmWorkspace& w, bool backward, cudaStream_t s) {
  const cudaError_t e = ssm_type(dt, [&](auto it) {
    using IT = decltype(it);
    return ssm_lanes(d.N, [&](auto nl) {
      constexpr int NL = decltype(nl)::value;
      const dim3 grid(fwd_blocks(d), unit_rows(d));
      if (backward)
        ssm_scan_kernel<IT, NL, kStartGrad><<<grid, fwd_threads(NL), 0, s>>>(
            d, (const IT*)in.dy, d.ld_dy, (const IT*)in.dt, in.A, (const IT*)in.Cm, d.ld_c, nullptr, nullptr, in.dt_bias,
            nullptr, 0, nullptr, nullptr, nullptr, w.R, w.sum_delta);
      else
        ssm_scan_kernel<IT, NL, kEndState><<<grid, fwd_threads(NL), 0, s>>>(
            d, (const IT*)in.x, d.ld_x, (const IT*)in.dt, in.A, (const IT*)in.Bm, d.ld_b, nullptr, nullptr, in.dt_bias,
            nullptr, 0, nullptr, nullptr, nullptr, w.R, w.sum_delta);
      stage_mark(s, backward ? "ssm_bwd_segments" : "ssm_fwd_segments");
      return cudaGetLastError();
    });
  });
  if (e != cudaSuccess) return e;
  const long long n = (long long)d.num_seqs * d.D * d.N;
  ssm_join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(d, in.A, edge, w.R, w.sum_delta, backward);
  stage_mark(s, "ssm_join");
  return cudaGetLastError();
}

}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_ssm_saved_bytes(const gdr_ssm_problem* p) {
  SsmDims d;
  return resolve_ssm(p, false, &d) == GDR_OK ? sizeof(float) * (size_t)d.max_tiles * d.D * d.N : 0;
}

size_t gdr_ssm_fwd_workspace_bytes(const gdr_ssm_problem* p) {
  SsmDims d;
  return resolve_ssm(p, false, &d) == GDR_OK ? ssm_workspace(d, nullptr, false).bytes : 0;
}

gdr_status gdr_ssm_fwd(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                       const void* Cm, const float* Dskip, const float* dt_bias, const float* S0, void* y, float* S_T,
                       float* h_saved, void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  SsmDims d;
  const gdr_status st = resolve_ssm(p, false, &d);
  if (st != GDR_OK) return st;
  if (!A || (d.total > 0 && (!x || !dt || !Bm || !Cm || !y))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(x, el) || !elem_ok(dt, el) || !elem_ok(Bm, el) || !elem_ok(Cm, el) || !elem_ok(y, el) || !vec_ok(A) ||
      !elem_ok(Dskip, 4) || !elem_ok(dt_bias, 4) || !vec_ok(S0) || !vec_ok(S_T) || !vec_ok(h_saved) || !elem_ok(d.cu, 4) ||
      ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  const SsmWorkspace w = ssm_workspace(d, (char*)workspace, false);
  if (!workspace || workspace_bytes < w.bytes) return GDR_ERR_WORKSPACE;
  if (d.num_seqs == 0) return GDR_OK;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  cudaError_t e = ssm_launch_index(&d, w, s);
  if (e != cudaSuccess) return status_of(e);
  const bool split = ssm_split(d);
  if (split) {
    const SsmInputs in{x, dt, Bm, Cm, nullptr, A, Dskip, dt_bias};
    e = ssm_launch_boundaries(d, p->dtype, in, S0, w, false, s);
    if (e != cudaSuccess) return status_of(e);
  }
  return status_of(ssm_type(p->dtype, [&](auto it) {
    using IT = decltype(it);
    return ssm_lanes(d.N, [&](auto nl) {
      constexpr int NL = decltype(nl)::value;
      ssm_scan_kernel<IT, NL, kFull><<<dim3(fwd_blocks(d), unit_rows(d)), fwd_threads(NL), 0, s>>>(
          d, (const IT*)x, d.ld_x, (const IT*)dt, A, (const IT*)Bm, d.ld_b, (const IT*)Cm, Dskip, dt_bias,
          split ? w.R : S0, split ? 1 : 0, (IT*)y, S_T, h_saved, nullptr, nullptr);
      stage_mark(s, "ssm_fwd");
      return cudaGetLastError();
    });
  }));
}

gdr_status gdr_ssm_step(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* Dskip, const float* dt_bias, float* pool, const int32_t* slots,
                        void* y, gdr_stream_t stream) {
  SsmDims d;
  const gdr_status st = resolve_ssm(p, true, &d);
  if (st != GDR_OK) return st;
  if (d.total == 0) return GDR_OK;
  if (!A || !x || !dt || !Bm || !Cm || !y || (!pool && p->num_slots > 0)) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(x, el) || !elem_ok(dt, el) || !elem_ok(Bm, el) || !elem_ok(Cm, el) || !elem_ok(y, el) || !vec_ok(A) ||
      !elem_ok(Dskip, 4) || !elem_ok(dt_bias, 4) || !vec_ok(pool) || !elem_ok(slots, 4))
    return GDR_ERR_ALIGNMENT;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  const long long grid = (d.total * d.D * (d.N / 4) + 255) / 256;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  return status_of(ssm_type(p->dtype, [&](auto it) {
    using IT = decltype(it);
    return ssm_lanes(d.N, [&](auto nl) {
      ssm_step_kernel<IT, decltype(nl)::value><<<(unsigned)grid, 256, 0, s>>>(
          d, p->B, p->num_slots, (const IT*)x, (const IT*)dt, A, (const IT*)Bm, (const IT*)Cm, Dskip, dt_bias, pool, slots,
          (IT*)y);
      stage_mark(s, "ssm_step");
      return cudaGetLastError();
    });
  }));
}

}  // extern "C"
