// gdr_ssm_bwd.cu -- backward of the selective state space scan (include/gdr_block.h):
//
//   dh_t = C_t dy_t + a_{t+1} dh_{t+1} (dS_T behind the last),   l_t = a_t dh_t h_{t-1},
//   dA = sum_t l_t D_t,   dD_t = sum_n l_t A + x_t s_t,  s_t = sum_n dh_t B_t,   dx_t = D_t s_t + Dskip dy_t,
//   dB_t = sum_d dh_t D_t x_t,   dC_t = sum_d dy_t h_t,   ddt = dD_t softplus'(dt + dt_bias),   dS0 = a_0 dh_0.
//
// A block walks its units' tiles of 16 tokens from the last to the first.  The forward left the
// state at the start of every tile, so the tile's states and decays are formed again in registers and
// then used in reverse.  Two states, or for the sums over channels two channels, share a register pair
// for the packed fp32 instructions.  Sums: over n across the lanes of a channel pair and over the
// channels of a warp, by exchanges that halve the values a lane keeps; over warps in shared memory;
// over blocks by a second kernel from per-block partial rows, in order: results do not depend on timing.
// Bound by instruction issue and the return path of shared-memory loads together: B = 2, T = 4096,
// D = 4096, N = 16, bf16: 479 us in this kernel (612 with two states per thread; 770 with the inputs'
// loads in registers as well; 1020 with separate instructions).
#include "gdr_ssm.cuh"

namespace gdr {
namespace {

// States per thread: two, or four.  With four what a token needs from shared memory serves eight states
// of the two channels, and a tile's states and decays fit the registers in two halves, for a second
// forward sweep over the first.  Both directions at B = 2, T = 4096, D = 2048, bf16, with two / four:
//   N = 8: 351 / 541 us  (a channel pair's shared memory then serves too few threads)
//   N = 16: 534 / 456 us, N = 32: 945 / 841 us, N = 64: 2008 / 1686 us
constexpr int bwd_states(int N) { return N >= 16 ? 4 : 2; }
constexpr int bwd_threads(int N) { return N == 4 ? 64 : N <= 16 ? 128 : 256; }

struct SsmBwdArgs {
  const void *x, *dt, *Bm, *Cm, *dy;
  const float *A, *Dskip, *dt_bias, *h_saved, *edge;
  int edge_per_unit;
  void *dx, *ddt;
  float *dS0, *grads, *bc;
};

// Shared memory of a block, two tiles of everything: the one being computed and the one that is
// formed (or finished) beside it.
template <typename IT, int N>
struct BwdSmem {
  static constexpr int NT = bwd_threads(N), S = bwd_states(N), ML = N / S, CB = 2 * NT / ML, WARPS = NT / 32;
  static constexpr int QP = 4 * CB > NT ? 4 * CB / NT : 1;  // quads of channels of a tile per thread
  // what a thread's own copies bring: its quads of dt, dy of the next tile; of x, which the tile's end
  // needs again, and its states, of three tiles
  Raw4<IT> raw[2][2][QP][NT], x[3][QP][NT];
  struct alignas(4 * S) Own {
    float v[S];
  } h[3][2][NT];
  Pair2 du[2][kTile][CB / 2];                      // {D, D'}, {D x, D' x'} of a channel pair
  f32x2 dy[2][kTile][CB / 2];
  alignas(16) float sig[2][kTile][CB];
  // sum_n dh B and sum_n l A; padded for the stores of a warp's lanes
  static constexpr int SR = CB + 8, SN = kTile * SR + 16;
  alignas(16) float s[2][2][SN];
  alignas(16) float B[2][kTile][N], C[2][kTile][N];
  float red[2][WARPS][kTile][2 * N];                     // dB, dC of a warp's channels
};

template <typename IT, int N>
__global__ void __launch_bounds__(bwd_threads(N), 256 / bwd_threads(N)) ssm_bwd_kernel(SsmDims d, SsmBwdArgs a) {
  using Smem = BwdSmem<IT, N>;
  constexpr int NT = Smem::NT, S = Smem::S, SP = S / 2, ML = Smem::ML, CB = Smem::CB, WARPS = Smem::WARPS, CL = 32 / ML;
  constexpr int kHalf = S == 2 ? kTile : kTile / 2;  // tokens whose states are kept at a time
  constexpr int Q = CB / 4, QP = Smem::QP;  // quads of channels; of a tile per thread
  constexpr int BQ = (8 * N + NT - 1) / NT;                      // quads of B and C per thread
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  if (ssm_bad(d)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nl = tid % ML, cl = lane / ML, pr = tid / ML;  // states S nl .. S nl + S - 1 of channel pair pr
  const int blocks = (d.Dg + CB - 1) / CB, grp = blockIdx.x / blocks, blk = blockIdx.x - grp * blocks, c0 = blk * CB;
  const int nch = min(CB, d.Dg - c0);
  const long long dc0 = (long long)grp * d.Dg + c0;
  const bool live[2] = {2 * pr < nch, 2 * pr + 1 < nch};
  const long long dch = dc0 + 2 * pr;
  // [channel][pair of states]; a missing channel has A = 0 and loads zeros
  using States = f32x2[2][SP];
  using Own = typename Smem::Own;
  auto unpack = [&](const Own(&o)[2], States& v) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < SP; ++j) v[c][j] = pack2(o[c].v[2 * j], o[c].v[2 * j + 1]);
  };
  auto load_states = [&](const float* p, States& v) {  // p: [D][N]
    Own o[2] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (live[c]) o[c] = *reinterpret_cast<const Own*>(p + (dch + c) * N + S * nl);
    unpack(o, v);
  };
  States A1, A2, dA = {};
  load_states(a.A, A1);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int j = 0; j < SP; ++j) A2[c][j] = pack2(decay_rate(lo2(A1[c][j])), decay_rate(hi2(A1[c][j])));
  float dDs[4] = {}, dbias[4] = {};
  const int qc = 4 * (tid % Q), qt = tid / Q, qn = qt < kTile ? nch - qc : 0;
  float bias[4] = {}, skip[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a.dt_bias && i < qn) bias[i] = a.dt_bias[dc0 + qc + i];
    if (a.Dskip && i < qn) skip[i] = a.Dskip[dc0 + qc + i];
  }
  const bool vec = d.vec & 1, vec_bc = d.vec & 2;

  const long long units = ssm_unit_count(d);
  for (long long un = blockIdx.y; un < units; un += gridDim.y) {
    const SsmUnit q = ssm_unit(d, un);
    States dh = {};
    if (a.edge) load_states(a.edge + (a.edge_per_unit ? un : q.seq) * (long long)d.D * N, dh);
    const int tiles = (q.len + kTile - 1) / kTile;
    const IT* xq = (const IT*)a.x + (long long)q.t0 * d.ld_x + dc0 + qc;
    const IT* dq = (const IT*)a.dt + (long long)q.t0 * d.ld_dt + dc0 + qc;
    const IT* yq = (const IT*)a.dy + (long long)q.t0 * d.ld_dy + dc0 + qc;
    Raw4<IT> rb[BQ];
    // Step k works on tile tiles - 1 - k; whole: its 16 tokens and CB channels all exist, aligned.
    // The copies go straight to shared memory: as register loads they were put off to the end of the
    // computation they were to overlap with, there being no registers to hold them.
    auto whole = [&](int k) { return vec && nch == CB && (tiles - k) * kTile <= q.len; };
    auto fetch = [&](int k) {
      const int base = (tiles - 1 - k) * kTile;
      const float* hs = a.h_saved + ((q.tile0 + tiles - 1 - k) * d.D + dch) * N + S * nl;
      copy_async<4 * S>(&sm.h[k % 3][0][tid], live[0] ? hs : a.h_saved, live[0] ? 4 * S : 0);
      copy_async<4 * S>(&sm.h[k % 3][1][tid], live[1] ? hs + N : a.h_saved, live[1] ? 4 * S : 0);
      Raw4<IT>(*raw)[QP][NT] = sm.raw[k & 1];
      if (whole(k)) {
#pragma unroll
        for (int i = 0; i < QP; ++i) {
          const long long t = base + qt + i * (NT / Q);
          if (qt < kTile) {
            copy_async<sizeof(Raw4<IT>)>(&sm.x[k % 3][i][tid], xq + t * d.ld_x, sizeof(Raw4<IT>));
            copy_async<sizeof(Raw4<IT>)>(&raw[0][i][tid], dq + t * d.ld_dt, sizeof(Raw4<IT>));
            copy_async<sizeof(Raw4<IT>)>(&raw[1][i][tid], yq + t * d.ld_dy, sizeof(Raw4<IT>));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < QP; ++i) {
          const long long t = base + qt + i * (NT / Q);
          const int n = t < q.len ? qn : 0;
          sm.x[k % 3][i][tid] = load_raw4(xq + t * d.ld_x, n, vec);
          raw[0][i][tid] = load_raw4(dq + t * d.ld_dt, n, vec);
          raw[1][i][tid] = load_raw4(yq + t * d.ld_dy, n, vec);
        }
      }
#pragma unroll
      for (int i = 0; i < BQ; ++i) {
        const int e = i * NT + tid, w = e % (4 * N), t = base + w / (N / 4), n = 4 * (w % (N / 4));
        if (e < 8 * N) {
          const IT* p = e < 4 * N ? (const IT*)a.Bm + (q.t0 + (long long)t) * d.ld_b : (const IT*)a.Cm + (q.t0 + (long long)t) * d.ld_c;
          rb[i] = load_raw4(p + (long long)grp * N + n, t < q.len ? 4 : 0, vec_bc);
        }
      }
    };
    auto form = [&](int k) {
      const int base = (tiles - 1 - k) * kTile, buf = k & 1;
      const bool full = whole(k);
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        const int tt = qt + i * (NT / Q);
        if (qt < kTile) {
          float xv[4], dv[4], yv[4], sg[4] = {1.f, 1.f, 1.f, 1.f};
          sm.x[k % 3][i][tid].get(xv);
          sm.raw[buf][0][i][tid].get(dv);
          sm.raw[buf][1][i][tid].get(yv);
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            f32x2 dl = add2(pack2(dv[c], dv[c + 1]), pack2(bias[c], bias[c + 1]));
            if (d.softplus) dl = softplus2(lo2(dl), hi2(dl), &sg[c], &sg[c + 1]);
            if (!full) {  // past the end nothing moves
              const int n = base + tt < q.len ? qn : 0;
              dl = pack2(c < n ? lo2(dl) : 0.f, c + 1 < n ? hi2(dl) : 0.f);
              if (c >= n) sg[c] = 0.f;
              if (c + 1 >= n) sg[c + 1] = 0.f;
            }
            sm.du[buf][tt][(qc + c) / 2] = Pair2{dl, mul2(dl, pack2(xv[c], xv[c + 1]))};
          }
          *reinterpret_cast<float4*>(&sm.dy[buf][tt][qc / 2]) = make_float4(yv[0], yv[1], yv[2], yv[3]);
          *reinterpret_cast<float4*>(&sm.sig[buf][tt][qc]) = make_float4(sg[0], sg[1], sg[2], sg[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < BQ; ++i) {
        const int e = i * NT + tid, w = e % (4 * N), t = w / (N / 4), n = 4 * (w % (N / 4));
        if (e < 8 * N) {
          float v[4];
          rb[i].get(v);
          *reinterpret_cast<float4*>(e < 4 * N ? &sm.B[buf][t][n] : &sm.C[buf][t][n]) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    };
    // what leaves from step k: dx, ddt of this thread's quads, dB and dC of the block
    auto finish = [&](int k) {
      const int base = (tiles - 1 - k) * kTile, buf = k & 1;
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        const int tt = qt + i * (NT / Q), t = base + tt;
        if (qt < kTile && t < q.len) {
          const float4 s1 = *reinterpret_cast<const float4*>(&sm.s[buf][0][tt * Smem::SR + qc]);
          const float4 s2 = *reinterpret_cast<const float4*>(&sm.s[buf][1][tt * Smem::SR + qc]);
          const float4 g4 = *reinterpret_cast<const float4*>(&sm.sig[buf][tt][qc]);
          const float4 y4 = *reinterpret_cast<const float4*>(&sm.dy[buf][tt][qc / 2]);
          const f32x2 d0 = sm.du[buf][tt][qc / 2].a, d1 = sm.du[buf][tt][qc / 2 + 1].a;
          const float s1v[4] = {s1.x, s1.y, s1.z, s1.w}, s2v[4] = {s2.x, s2.y, s2.z, s2.w};
          float xv[4];
          sm.x[k % 3][i][tid].get(xv);
          const float gv[4] = {g4.x, g4.y, g4.z, g4.w}, yv[4] = {y4.x, y4.y, y4.z, y4.w};
          const float dl[4] = {lo2(d0), hi2(d0), lo2(d1), hi2(d1)};
          float ox[4], og[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ox[c] = fmaf(s1v[c], dl[c], skip[c] * yv[c]);
            og[c] = fmaf(s1v[c], xv[c], s2v[c]) * gv[c];
            dDs[c] = fmaf(yv[c], xv[c], dDs[c]);
            dbias[c] += og[c];
          }
          const long long at = (long long)(q.t0 + t) * d.D + dc0 + qc;
          store4((IT*)a.dx + at, qn, vec, ox);
          store4((IT*)a.ddt + at, qn, vec, og);
        }
      }
#pragma unroll 2
      for (int e = tid; e < kTile * N / 2; e += NT) {  // four sums each
        const int t = e / (N / 2), v = 4 * (e % (N / 2));
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float4 r = *reinterpret_cast<const float4*>(&sm.red[buf][w][t][v]);
          s.x += r.x; s.y += r.y; s.z += r.z; s.w += r.w;
        }
        if (base + t < q.len)
          *reinterpret_cast<float4*>(a.bc + (((long long)blk * d.total + q.t0 + base + t) * d.G + grp) * 2 * N + v) = s;
      }
    };
    if (tiles > 0) {
      fetch(0);
      copy_async_wait();
      form(0);
      if (tiles > 1) fetch(1);
    }
    for (int k = 0; k < tiles; ++k) {
      const int buf = k & 1;
      copy_async_wait();  // the copies of tile k + 1, a whole tile's work ago
      __syncthreads();
      if (k > 0) finish(k - 1);  // before form overwrites this thread's own entries of that tile
      if (k + 1 < tiles) form(k + 1);
      if (k + 2 < tiles) fetch(k + 2);
      States h0;  // in front of the tile
      {
        const Own o[2] = {sm.h[k % 3][0][tid], sm.h[k % 3][1][tid]};
        unpack(o, h0);
      }
      struct alignas(8 * SP) Some {
        f32x2 v[SP];
      };
      struct Operands {
        Pair2 du;
        Some b, c;
        f32x2 dy;
      };
      auto load_db = [&](int t, Operands& o) {
        o.du = sm.du[buf][t][pr];
        o.b = *reinterpret_cast<const Some*>(&sm.B[buf][t][S * nl]);
      };
      auto load_cy = [&](int t, Operands& o) {
        o.c = *reinterpret_cast<const Some*>(&sm.C[buf][t][S * nl]);
        o.dy = sm.dy[buf][t][pr];
      };
      auto both = [](f32x2 v, int c) { return c ? pack2(hi2(v), hi2(v)) : pack2(lo2(v), lo2(v)); };
      // from the state in front of token t to the one behind it; e: the decays
      auto advance = [&](const Operands& o, const States& from, States& to, States& e) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const f32x2 dd = both(o.du.a, c), uu = both(o.du.b, c);
#pragma unroll
          for (int j = 0; j < SP; ++j) {
            e[c][j] = ex2_2(mul2(dd, A2[c][j]));
            to[c][j] = fma2(e[c][j], from[c][j], mul2(uu, o.b.v[j]));
          }
        }
      };
      States dAt = {};  // a tile's part first: the long sum then has 1/16 of the terms
      // kHalf tokens: their states and decays in order, then their gradients in reverse
      auto half = [&](int first, const States& from) {
        States h[kHalf + 1], e[kHalf];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < SP; ++j) h[0][c][j] = from[c][j];
        Operands nx;  // a token's operands are loaded a token ahead
        load_db(first, nx);
#pragma unroll
        for (int t = 0; t < kHalf; ++t) {
          const Operands o = nx;
          if (t + 1 < kHalf) load_db(first + t + 1, nx);
          advance(o, h[t], h[t + 1], e[t]);
        }
        load_cy(first + kHalf - 1, nx);
#pragma unroll
        for (int t2 = kHalf - 2; t2 >= 0; t2 -= 2) {
          float s[8];  // {s1, s1', s2, s2'} of tokens t2, t2 + 1
#pragma unroll
          for (int i = 1; i >= 0; --i) {
            const int t = t2 + i;
            const Operands o = nx;
            if (t > 0) {
              load_db(first + t - 1, nx);
              load_cy(first + t - 1, nx);
            }
            f32x2 wb[SP], wc[SP];  // this pair's part of dB and dC of the states
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const f32x2 dd = both(o.du.a, c), uu = both(o.du.b, c), yy = both(o.dy, c);
              f32x2 s1, s2;
#pragma unroll
              for (int j = 0; j < SP; ++j) {
                dh[c][j] = fma2(yy, o.c.v[j], dh[c][j]);
                wb[j] = c ? fma2(dh[c][j], uu, wb[j]) : mul2(dh[c][j], uu);
                wc[j] = c ? fma2(yy, h[t + 1][c][j], wc[j]) : mul2(yy, h[t + 1][c][j]);
                s1 = j ? fma2(dh[c][j], o.b.v[j], s1) : mul2(dh[c][j], o.b.v[j]);
                dh[c][j] = mul2(dh[c][j], e[t][c][j]);
                const f32x2 l = mul2(dh[c][j], h[t][c][j]);
                s2 = j ? fma2(l, A1[c][j], s2) : mul2(l, A1[c][j]);
                dAt[c][j] = fma2(l, dd, dAt[c][j]);
              }
              s[4 * i + c] = lo2(s1) + hi2(s1);
              s[4 * i + 2 + c] = lo2(s2) + hi2(s2);
            }
            float w[2 * S];
#pragma unroll
            for (int j = 0; j < SP; ++j) {
              w[2 * j] = lo2(wb[j]);
              w[2 * j + 1] = hi2(wb[j]);
              w[S + 2 * j] = lo2(wc[j]);
              w[S + 2 * j + 1] = hi2(wc[j]);
            }
            using Chan = LaneSums<2 * S, CL, ML>;  // over the warp's channel pairs
            Chan::run(w, cl);
            if (Chan::holds(cl)) {
#pragma unroll
              for (int v = 0; v < Chan::KEEP; ++v) {
                const int vi = Chan::index(cl) + v;  // dB of states S nl .., then dC
                sm.red[buf][warp][first + t][(vi / S) * N + S * nl + vi % S] = w[v];
              }
            }
          }
          using Stat = LaneSums<8, ML, 1>;  // over the states
          Stat::run(s, nl);
          if (Stat::holds(nl)) {
#pragma unroll
            for (int v = 0; v < Stat::KEEP; ++v) {
              const int vi = Stat::index(nl) + v;
              sm.s[buf][(vi >> 1) & 1][(first + t2 + (vi >> 2)) * Smem::SR + 2 * pr + (vi & 1)] = s[v];
            }
          }
        }
      };
      if constexpr (kHalf < kTile) {
        static_assert(kHalf % 2 == 0, "the state in front of the second half ends in at[0]");
        States at[2], e;  // turn about
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < SP; ++j) at[0][c][j] = h0[c][j];
        Operands nx;
        load_db(0, nx);
#pragma unroll
        for (int t = 0; t < kHalf; ++t) {
          const Operands o = nx;
          if (t + 1 < kHalf) load_db(t + 1, nx);
          advance(o, at[t & 1], at[(t + 1) & 1], e);
        }
        // one copy of the code for both halves (two overflow the instruction cache: 506 us for 479)
#pragma unroll 1
        for (int first = kHalf; first >= 0; first -= kHalf) {
          half(first, at[0]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < SP; ++j) at[0][c][j] = h0[c][j];
        }
      } else {
        half(0, h0);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < SP; ++j) dA[c][j] = add2(dA[c][j], dAt[c][j]);
    }
    __syncthreads();
    if (tiles > 0) finish(tiles - 1);
    if (a.dS0 && q.first) {
      float* o = a.dS0 + ((long long)q.seq * d.D + dch) * N + S * nl;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (live[c]) {
          Own v;
#pragma unroll
          for (int j = 0; j < SP; ++j) {
            v.v[2 * j] = lo2(dh[c][j]);
            v.v[2 * j + 1] = hi2(dh[c][j]);
          }
          *reinterpret_cast<Own*>(o + c * N) = v;
        }
    }
    __syncthreads();  // the next unit's first tile overwrites what finish read
  }
  // this row's sums over tokens: [N][D] of dA, [D] of dDskip, [D] of ddt_bias
  float* out = a.grads + (long long)blockIdx.y * (N + 2) * d.D;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (live[c])
#pragma unroll
      for (int j = 0; j < SP; ++j) {
        out[(long long)(S * nl + 2 * j) * d.D + dch + c] = lo2(dA[c][j]);
        out[(long long)(S * nl + 2 * j + 1) * d.D + dch + c] = hi2(dA[c][j]);
      }
  // dDskip, ddt_bias: over the threads that held the same channels
  __syncthreads();
  float* cols = reinterpret_cast<float*>(smem_raw);  // [NT][8]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cols[tid * 8 + i] = dDs[i];
    cols[tid * 8 + 4 + i] = dbias[i];
  }
  __syncthreads();
  for (int c = tid; c < 2 * CB; c += NT) {
    const int m = c / CB, cc = c - m * CB;
    float s = 0.f;
    for (int r = 0; r < NT / Q; ++r) s += cols[(r * Q + cc / 4) * 8 + 4 * m + (cc & 3)];
    if (cc < nch) out[(long long)(N + m) * d.D + dc0 + cc] = s;
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

// Calls f(N).
template <typename F>
cudaError_t ssm_states(int N, F f) {
  return ssm_lanes(N, [&](auto nl) { return f(std::integral_constant<int, 4 * decltype(nl)::value>{}); });
}

}  // namespace

int ssm_bwd_channels(int N) { return 2 * bwd_threads(N) / (N / bwd_states(N)); }

int ssm_bwd_rows(const SsmDims& d) {
  const int cb = ssm_bwd_channels(d.N);
  const long long blocks = (long long)d.G * ((d.Dg + cb - 1) / cb), most = (8 * kSmCount + blocks - 1) / blocks;
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
  d.vec = ssm_vec(d, el, {x, dt, dy, dx, ddt}, {Bm, Cm});
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
    cudaError_t r = ssm_states(d.N, [&](auto n) {
      constexpr int N = decltype(n)::value;
      constexpr size_t smem = sizeof(BwdSmem<IT, N>);
      static_assert(smem <= 227 * 1024, "shared memory of a block");
      const cudaError_t se = set_smem_once((const void*)ssm_bwd_kernel<IT, N>, smem);
      if (se != cudaSuccess) return se;
      ssm_bwd_kernel<IT, N><<<dim3((unsigned)(d.G * blocks), (unsigned)rows), bwd_threads(N), smem, s>>>(d, a);
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
