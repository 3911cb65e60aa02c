// gdr_ssm_bwd.cu -- backward of the selective state space scan (include/gdr_block.h):
//
//   dh_t = C_t dy_t + a_{t+1} dh_{t+1} (dS_T behind the last),   l_t = a_t dh_t h_{t-1},
//   dA = sum_t l_t D_t,   dD_t = sum_n l_t A + x_t s_t,  s_t = sum_n dh_t B_t,   dx_t = D_t s_t + Dskip dy_t,
//   dB_t = sum_d dh_t D_t x_t,   dC_t = sum_d dy_t h_t,   ddt = dD_t softplus'(dt + dt_bias),   dS0 = a_0 dh_0.
//
// A block walks its units' tiles of 16 tokens from the last to the first.  The forward left the
// state at the start of every tile, so the tile's 16 states are formed again in registers (16 x 4
// per thread) and then used in reverse; the decays are formed again too (an exponential costs less
// than 64 more registers).  Sums: over n across the lanes of a channel, over the channels of a warp
// by exchanges that halve the values a lane keeps, over warps in shared memory, over blocks by a
// second kernel from per-block partial rows in order, so results do not depend on timing.
#include "gdr_ssm.cuh"

namespace gdr {
namespace {

constexpr int bwd_threads(int NL) { return NL == 1 ? 64 : NL == 2 ? 128 : 256; }

struct SsmBwdArgs {
  const void *x, *dt, *Bm, *Cm, *dy;
  const float *A, *Dskip, *dt_bias, *h_saved, *edge;
  int edge_per_unit;
  void *dx, *ddt;
  float *dS0, *grads, *bc;
};

template <typename IT, int NL>
__global__ void __launch_bounds__(bwd_threads(NL), 1) ssm_bwd_kernel(SsmDims d, SsmBwdArgs a) {
  constexpr int NT = bwd_threads(NL), CB = NT / NL, N = 4 * NL, WARPS = NT / 32, CL = 32 / NL;
  constexpr int PER = kTile * CB / NT, PB = (kTile * N + NT - 1) / NT;
  extern __shared__ __align__(16) float smem[];
  float(*sd)[CB] = reinterpret_cast<float(*)[CB]>(smem);                // D_t
  float(*sx)[CB] = sd + kTile;                                          // x_t, then ddt
  float(*sy)[CB] = sx + kTile;                                          // dy_t, then dx
  float(*sg)[CB] = sy + kTile;                                          // softplus' (0 past the end)
  float(*sB)[N] = reinterpret_cast<float(*)[N]>(sg + kTile);
  float(*sC)[N] = sB + kTile;
  float* red = reinterpret_cast<float*>(sC + kTile);                    // [WARPS][16][2 N]
  if (ssm_bad(d)) return;
  const int tid = threadIdx.x, ln = tid % NL, ch = tid / NL, lane = tid & 31, warp = tid >> 5, cl = lane / NL;
  const int blocks = (d.Dg + CB - 1) / CB, grp = blockIdx.x / blocks, blk = blockIdx.x - grp * blocks, c0 = blk * CB;
  const int nch = min(CB, d.Dg - c0);
  const long long dc0 = (long long)grp * d.Dg + c0;
  const bool live = ch < nch;
  const long long dch = dc0 + ch;
  float A1[4] = {}, A2[4] = {};
  if (live) {
    const float4 v = *reinterpret_cast<const float4*>(a.A + dch * N + 4 * ln);
    A1[0] = v.x; A1[1] = v.y; A1[2] = v.z; A1[3] = v.w;
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] = fmaxf(A1[j] * kLog2e, -kBig);
  }
  const float skip = a.Dskip && live ? a.Dskip[dch] : 0.f;
  float dA[4] = {}, dDs = 0.f, dbias = 0.f;
  const IT *x = (const IT*)a.x, *dt = (const IT*)a.dt, *Bm = (const IT*)a.Bm, *Cm = (const IT*)a.Cm, *dy = (const IT*)a.dy;

  const long long units = ssm_unit_count(d);
  for (long long un = blockIdx.y; un < units; un += gridDim.y) {
    const SsmUnit q = ssm_unit(d, un);
    float dh[4] = {};
    if (a.edge && live) {
      const float4 v = *reinterpret_cast<const float4*>(a.edge + ((a.edge_per_unit ? un : q.seq) * d.D + dch) * N + 4 * ln);
      dh[0] = v.x; dh[1] = v.y; dh[2] = v.z; dh[3] = v.w;
    }
    const int tiles = (q.len + kTile - 1) / kTile;
    IT px[PER], pd[PER], py[PER], pB[PB], pC[PB];
    float4 ph = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fetch = [&](int tile) {
      const int base = tile * kTile;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * NT + tid, t = base + e / CB, c = e % CB;
        const bool in = t < q.len && c < nch;
        const long long tok = q.t0 + t;
        px[i] = in ? x[tok * d.ld_x + dc0 + c] : from_f32<IT>(0.f);
        pd[i] = in ? dt[tok * d.ld_dt + dc0 + c] : from_f32<IT>(0.f);
        py[i] = in ? dy[tok * d.ld_dy + dc0 + c] : from_f32<IT>(0.f);
      }
#pragma unroll
      for (int i = 0; i < PB; ++i) {
        const int e = i * NT + tid, t = base + e / N, n = e % N;
        const bool in = e < kTile * N && t < q.len;
        pB[i] = in ? Bm[(long long)(q.t0 + t) * d.ld_b + grp * N + n] : from_f32<IT>(0.f);
        pC[i] = in ? Cm[(long long)(q.t0 + t) * d.ld_c + grp * N + n] : from_f32<IT>(0.f);
      }
      if (live) ph = *reinterpret_cast<const float4*>(a.h_saved + ((q.tile0 + tile) * d.D + dch) * N + 4 * ln);
    };
    if (tiles > 0) fetch(tiles - 1);
    for (int tile = tiles - 1; tile >= 0; --tile) {
      const int base = tile * kTile;
      __syncthreads();  // the previous tile's readers are done
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * NT + tid, t = e / CB, c = e % CB;
        const bool in = base + t < q.len && c < nch;
        float raw = to_f32(pd[i]), dl = 0.f, sig = 0.f;
        if (in) {
          if (a.dt_bias) raw += a.dt_bias[dc0 + c];
          dl = raw;
          sig = 1.f;
          if (d.softplus) dl = softplus_f(raw, &sig);
        }
        sd[t][c] = dl;
        sg[t][c] = sig;
        sx[t][c] = to_f32(px[i]);
        sy[t][c] = to_f32(py[i]);
      }
#pragma unroll
      for (int i = 0; i < PB; ++i) {
        const int e = i * NT + tid;
        if (e < kTile * N) {
          sB[e / N][e % N] = to_f32(pB[i]);
          sC[e / N][e % N] = to_f32(pC[i]);
        }
      }
      float h[kTile + 1][4];  // h[t]: the state in front of token t
      h[0][0] = ph.x; h[0][1] = ph.y; h[0][2] = ph.z; h[0][3] = ph.w;
      __syncthreads();
      if (tile > 0) fetch(tile - 1);
#pragma unroll
      for (int t = 0; t < kTile; ++t) {
        const float dl = sd[t][ch], u = dl * sx[t][ch];
        const float4 b = *reinterpret_cast<const float4*>(&sB[t][4 * ln]);
        const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) h[t + 1][j] = fmaf(ex2f(dl * A2[j]), h[t][j], u * bb[j]);
      }
#pragma unroll
      for (int t4 = kTile - 4; t4 >= 0; t4 -= 4) {
        float s1[4], s2[4];  // sum_n dh B and sum_n l A of the four tokens
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          const int t = t4 + i;
          const float dl = sd[t][ch], u = dl * sx[t][ch], dyv = sy[t][ch];
          const float4 b = *reinterpret_cast<const float4*>(&sB[t][4 * ln]);
          const float4 c = *reinterpret_cast<const float4*>(&sC[t][4 * ln]);
          const float bb[4] = {b.x, b.y, b.z, b.w}, cc[4] = {c.x, c.y, c.z, c.w};
          float w[8];  // this channel's part of dB_t and dC_t
          s1[i] = s2[i] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dh[j] = fmaf(dyv, cc[j], dh[j]);
            w[j] = dh[j] * u;
            w[4 + j] = dyv * h[t + 1][j];
            s1[i] = fmaf(dh[j], bb[j], s1[i]);
            dh[j] *= ex2f(dl * A2[j]);
            const float l = dh[j] * h[t][j];
            s2[i] = fmaf(l, A1[j], s2[i]);
            dA[j] = fmaf(l, dl, dA[j]);
          }
          // over the warp's channels: value index bits 2, 1, 0 go to channel bits 0, 1, 2
#pragma unroll
          for (int bit = 0; (1 << bit) < CL; ++bit) {
            const int off = NL << bit, m = bit == 0 ? 4 : bit == 1 ? 2 : bit == 2 ? 1 : 0;
            if (m > 0) {
              const bool hi = cl & (1 << bit);
#pragma unroll
              for (int v = 0; v < m; ++v) {
                const float send = hi ? w[v] : w[v + m], keep = hi ? w[v + m] : w[v];
                w[v] = keep + __shfl_xor_sync(0xffffffffu, send, off);
              }
            } else {
              w[0] += __shfl_xor_sync(0xffffffffu, w[0], off);
            }
          }
          constexpr int KEEP = CL >= 8 ? 1 : 8 / CL;
          const int first = CL >= 8 ? (cl & 1) * 4 + ((cl >> 1) & 1) * 2 + ((cl >> 2) & 1)
                                    : CL == 4 ? (cl & 1) * 4 + ((cl >> 1) & 1) * 2 : CL == 2 ? (cl & 1) * 4 : 0;
          if (cl < 8)
#pragma unroll
            for (int v = 0; v < KEEP; ++v) {
              const int vi = first + v;  // dB of state 4 ln + vi, or dC of state 4 ln + vi - 4
              red[(warp * kTile + t) * 2 * N + (vi < 4 ? 0 : N) + 4 * ln + (vi & 3)] = w[v];
            }
        }
        LaneSum<NL>::run(s1, ln);
        LaneSum<NL>::run(s2, ln);
        if (LaneSum<NL>::holds(ln)) {
#pragma unroll
          for (int k = 0; k < LaneSum<NL>::kKeep; ++k) {
            const int t = t4 + LaneSum<NL>::tok(ln) + k;
            const float xv = sx[t][ch], dyv = sy[t][ch], g = fmaf(s1[k], xv, s2[k]) * sg[t][ch];
            dDs = fmaf(dyv, xv, dDs);
            dbias += g;
            sy[t][ch] = fmaf(s1[k], sd[t][ch], skip * dyv);
            sx[t][ch] = g;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * NT + tid, t = e / CB, c = e % CB;
        if (base + t < q.len && c < nch) {
          const long long at = (long long)(q.t0 + base + t) * d.D + dc0 + c;
          ((IT*)a.dx)[at] = from_f32<IT>(sy[t][c]);
          ((IT*)a.ddt)[at] = from_f32<IT>(sx[t][c]);
        }
      }
      for (int e = tid; e < kTile * 2 * N; e += NT) {
        const int t = e / (2 * N), v = e % (2 * N);
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += red[w * kTile * 2 * N + e];
        if (base + t < q.len)
          a.bc[(((long long)blk * d.total + q.t0 + base + t) * d.G + grp) * 2 * N + v] = s;
      }
    }
    if (a.dS0 && q.first && live)
      *reinterpret_cast<float4*>(a.dS0 + ((long long)q.seq * d.D + dch) * N + 4 * ln) = make_float4(dh[0], dh[1], dh[2], dh[3]);
  }
  // this row's sums over tokens: [N][D] of dA, [D] of dDskip, [D] of ddt_bias
  float* out = a.grads + (long long)blockIdx.y * (N + 2) * d.D;
#pragma unroll
  for (int o = 1; o < NL; o <<= 1) {
    dDs += __shfl_xor_sync(0xffffffffu, dDs, o);
    dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
  }
  if (live) {
#pragma unroll
    for (int j = 0; j < 4; ++j) out[(long long)(4 * ln + j) * d.D + dch] = dA[j];
    if (ln == 0) {
      out[(long long)N * d.D + dch] = dDs;
      out[(long long)(N + 1) * d.D + dch] = dbias;
    }
  }
}

// dB, dC of every token and group: the channel blocks' rows [blocks][tokens][G][2 N] added in order.
template <typename IT>
__global__ void __launch_bounds__(256) ssm_bc_kernel(SsmDims d, const float* __restrict__ bc, int blocks,
                                                     IT* __restrict__ dB, IT* __restrict__ dC) {
  if (ssm_bad(d)) return;
  const long long row = (long long)d.G * 2 * d.N, n = d.total * row;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int b = 0; b < blocks; ++b) s += bc[b * n + id];
  const long long tg = id / (2 * d.N);
  const int v = (int)(id - tg * 2 * d.N);
  if (v < d.N)
    dB[tg * d.N + v] = from_f32<IT>(s);
  else
    dC[tg * d.N + v - d.N] = from_f32<IT>(s);
}

size_t bwd_smem(int NL) {
  const int NT = bwd_threads(NL), CB = NT / NL, N = 4 * NL;
  return sizeof(float) * (size_t)(4 * kTile * CB + 2 * kTile * N + NT / 32 * kTile * 2 * N);
}

}  // namespace

int ssm_bwd_channels(int N) { return bwd_threads(N / 4) / (N / 4); }

int ssm_bwd_rows(const SsmDims& d) {
  const int cb = ssm_bwd_channels(d.N);
  const long long blocks = (long long)d.G * ((d.Dg + cb - 1) / cb), most = (4 * kSmCount + blocks - 1) / blocks;
  const long long rows = d.max_units < most ? d.max_units : most;
  return (int)(rows < 1 ? 1 : rows);
}

}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_ssm_bwd_workspace_bytes(const gdr_ssm_problem* p) {
  SsmDims d;
  return resolve_ssm(p, false, &d) == GDR_OK ? ssm_workspace(d, nullptr, true).bytes : 0;
}

gdr_status gdr_ssm_bwd(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                       const void* Cm, const float* Dskip, const float* dt_bias, const float* h_saved, const void* dy,
                       const float* dS_T, void* dx, void* ddt, float* dA, void* dBm, void* dCm, float* dDskip,
                       float* ddt_bias, float* dS0, void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  SsmDims d;
  const gdr_status st = resolve_ssm(p, false, &d);
  if (st != GDR_OK) return st;
  if (!A || !dA || (d.total > 0 && (!x || !dt || !Bm || !Cm || !dy || !h_saved || !dx || !ddt || !dBm || !dCm)))
    return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  const void* elems[] = {x, dt, Bm, Cm, dy, dx, ddt, dBm, dCm};
  const void* floats[] = {Dskip, dt_bias, dA, dDskip, ddt_bias, d.cu};
  for (const void* v : elems)
    if (!elem_ok(v, el)) return GDR_ERR_ALIGNMENT;
  for (const void* v : floats)
    if (!elem_ok(v, 4)) return GDR_ERR_ALIGNMENT;
  if (!vec_ok(A) || !vec_ok(h_saved) || !vec_ok(dS_T) || !vec_ok(dS0) || ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  const SsmWorkspace w = ssm_workspace(d, (char*)workspace, true);
  if (!workspace || workspace_bytes < w.bytes) return GDR_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  cudaError_t e = ssm_launch_index(&d, w, s);
  if (e != cudaSuccess) return status_of(e);
  const bool split = ssm_split(d);
  if (split) {
    const SsmInputs in{x, dt, Bm, Cm, dy, A, Dskip, dt_bias};
    e = ssm_launch_boundaries(d, p->dtype, in, dS_T, w, true, s);
    if (e != cudaSuccess) return status_of(e);
  }
  const int cb = ssm_bwd_channels(d.N), blocks = (d.Dg + cb - 1) / cb, rows = ssm_bwd_rows(d);
  const SsmBwdArgs a{x, dt, Bm, Cm, dy, A, Dskip, dt_bias, h_saved, split ? w.R : dS_T, split ? 1 : 0,
                     dx, ddt, dS0, w.grads, w.bc};
  auto run = [&](auto it) {
    using IT = decltype(it);
    cudaError_t r = ssm_lanes(d.N, [&](auto nl) {
      constexpr int NL = decltype(nl)::value;
      const size_t smem = bwd_smem(NL);
      const cudaError_t se = set_smem_once((const void*)ssm_bwd_kernel<IT, NL>, smem);
      if (se != cudaSuccess) return se;
      ssm_bwd_kernel<IT, NL><<<dim3((unsigned)(d.G * blocks), (unsigned)rows), bwd_threads(NL), smem, s>>>(d, a);
      stage_mark(s, "ssm_bwd");
      return cudaGetLastError();
    });
    if (r != cudaSuccess || d.total == 0) return r;
    const long long n = d.total * d.G * 2 * d.N, grid = (n + 255) / 256;
    if (grid >= (1ll << 31)) return cudaErrorInvalidConfiguration;
    ssm_bc_kernel<IT><<<(unsigned)grid, 256, 0, s>>>(d, w.bc, blocks, (IT*)dBm, (IT*)dCm);
    stage_mark(s, "ssm_bc");
    return cudaGetLastError();
  };
  e = p->dtype == GDR_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
  if (e != cudaSuccess) return status_of(e);
  ColumnSums out = {};
  out.mat = dA;
  out.mat_parts = d.N;
  out.vec[0] = dDskip;
  out.vec[1] = ddt_bias;
  out.parts = d.N + 2;
  out.width = d.D;
  out.status = d.status;
  return status_of(launch_column_sums(w.grads, rows, out, s, "ssm_dA"));
}

}  // extern "C"
