// gdr_ssm.cu -- the selective state space scan, forward and single token (include/gdr_block.h):
//
//   D_t = softplus(dt_t + dt_bias),  h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,  y_t = sum_n C_t h_t + Dskip x_t
//
// Every (channel, state) pair decays at a rate of its own, so there is no matrix product whose
// factors stay in range: the recurrence runs token by token in fp32 registers.  NL = N / 4 lanes
// share a channel, four states each; the sum over n runs over those lanes for four tokens at a
// time.  A block holds 64 channels; D_t, D_t x_t, B_t and C_t of 16 tokens are formed once per token
// and channel and staged in shared memory.  Not bound by memory from
// N = 8 on: per (token, channel, state) one exponential and four multiply-adds, against 6 / N bytes in
// bf16.  B = 2, T = 4096, D = 4096, N = 16: 166 us for the full pass (issue slots and the return path of
// shared-memory loads each about 0.62 used, at 16 warps per SM), 103 us for the first pass (the
// exponentials' unit at 0.56); the exponentials alone are 58 us a pass.
//
// Where the channels do not fill the GPU the sequence is cut into segments: a first pass finds
// every segment's end state from zero, a scan joins them (the decay over a segment is exp(A sum D_t),
// one exponential), and the full pass runs all segments side by side from their true states.
#include "gdr_ssm.cuh"

namespace gdr {
namespace {

// Threads of a block: 32 pairs of channels by the NL lanes of each.
constexpr int fwd_threads(int NL) { return 32 * NL; }
constexpr int kFwdChannels = 64;

enum SsmMode { kFull, kEndState, kStartGrad };

// kFull: y (and states, S_T).  kEndState: R[u] = end state of unit u from zero, and sum of D_t.
// kStartGrad (in reverse): R[u] = gradient of the state in front of unit u from a zero gradient
// behind it; x is dy, and C plays B's part.
//
// A thread holds two channels by four states.  What a token needs comes from shared memory in three
// 16-byte loads (the two channels' D and D x, four B, four C) for eight states: with one channel
// (and D, D x stored twice for the packed instructions) the loads' return path, 128 bytes a clock
// and SM, was the bound: 213 us at B = 1, T = 32768, D = 1024, N = 16.
//
// One barrier per tile: while tile k is computed from one buffer, tile k + 1 is formed in the other
// from registers that tile k + 2's loads then refill, and tile k - 1's y leaves.  A thread forms and
// finishes the same four channels of a token.
template <typename IT, int NL, int MODE>
__global__ void __launch_bounds__(fwd_threads(NL))
    ssm_scan_kernel(SsmDims d, const IT* __restrict__ x, long long ld_x, const IT* __restrict__ dt,
                    const float* __restrict__ A, const IT* __restrict__ Bm, long long ld_b,
                    const IT* __restrict__ Cm, const float* __restrict__ Dskip, const float* __restrict__ dt_bias,
                    const float* __restrict__ start, int start_per_unit, IT* __restrict__ y, float* __restrict__ S_T,
                    float* __restrict__ h_saved, float* __restrict__ R, float* __restrict__ sum_delta) {
  constexpr int NT = fwd_threads(NL), CB = kFwdChannels, PB = CB / 2, N = 4 * NL;
  constexpr int Q = CB / 4, QP = kTile * Q > NT ? kTile * Q / NT : 1;  // quads of channels; of a tile per thread
  constexpr int YS = CB + 16;
  constexpr bool kY = MODE == kFull;
  __shared__ Pair2 sdu[2][kTile][PB];  // {D, D'}, {D x, D' x'} of a channel pair, at slot(pair)
  __shared__ __align__(16) float sB[2][kTile][N], sC[kY ? 2 : 1][kTile][N];
  __shared__ __align__(16) float sy[kY ? 2 : 1][kY ? kTile : 1][YS];
  if (ssm_bad(d)) return;
  auto slot = [](int p) { return p ^ ((p >> 3) & 1); };  // a quad's two stores hit all banks
  const int tid = threadIdx.x, ln = tid % NL, pr = tid / NL;
  const int blocks = (d.Dg + CB - 1) / CB, grp = blockIdx.x / blocks, c0 = (blockIdx.x - grp * blocks) * CB;
  const int nch = min(CB, d.Dg - c0);                // live channels of this block
  const long long dc0 = (long long)grp * d.Dg + c0;  // its first channel
  const bool live[2] = {2 * pr < nch, 2 * pr + 1 < nch};
  const long long dch = dc0 + 2 * pr;
  auto load_state = [&](const float* p, f32x2 (&v)[2][2]) {  // p: [D][N]; a missing channel is zeros
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float4 f = live[c] ? *reinterpret_cast<const float4*>(p + (dch + c) * N + 4 * ln) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[c][0] = pack2(f.x, f.y);
      v[c][1] = pack2(f.z, f.w);
    }
  };
  auto store_state = [&](float* p, const f32x2 (&v)[2][2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (live[c])
        *reinterpret_cast<float4*>(p + (dch + c) * N + 4 * ln) = make_float4(lo2(v[c][0]), hi2(v[c][0]), lo2(v[c][1]), hi2(v[c][1]));
  };
  f32x2 A2[2][2];
  load_state(A, A2);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int j = 0; j < 2; ++j) A2[c][j] = pack2(decay_rate(lo2(A2[c][j])), decay_rate(hi2(A2[c][j])));
  // staging: quad of channels qc of token qt (+ NT / Q tokens per further quad)
  const int qc = 4 * (tid % Q), qt = tid / Q, qn = qt < kTile ? nch - qc : 0;
  float bias[4] = {}, skip[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dt_bias && i < qn) bias[i] = dt_bias[dc0 + qc + i];
    if (kY && Dskip && i < qn) skip[i] = Dskip[dc0 + qc + i];
  }
  const bool vec = d.vec & 1, vec_bc = d.vec & 2;
  const bool is_c = tid >= 4 * N, has_bc = tid < (kY ? 8 : 4) * N;  // one quad of B or C per thread
  const int bt = (tid % (4 * N)) / NL, bn = 4 * (tid % NL);
  const IT* bc_src = is_c ? Cm : Bm;
  const long long ld_bc = is_c ? d.ld_c : ld_b;

  const long long units = ssm_unit_count(d);
  for (long long un = blockIdx.y; un < units; un += gridDim.y) {
    const SsmUnit q = ssm_unit(d, un);
    // nothing follows a sequence's last unit (in reverse: its first) that its boundary would be for
    if (MODE == kEndState ? q.last : MODE == kStartGrad ? q.first : false) continue;
    f32x2 h[2][2] = {};
    if (kY && start) load_state(start + (start_per_unit ? un : q.seq) * (long long)d.D * N, h);
    f32x2 dsum = 0;
    const int tiles = (q.len + kTile - 1) / kTile;
    auto base_of = [&](int k) { return (MODE == kStartGrad ? tiles - 1 - k : k) * kTile; };
    // a tile whose 16 tokens and CB channels all exist, aligned: no bounds in its loads and stores
    auto whole = [&](int k) { return vec && nch == CB && base_of(k) + kTile <= q.len; };
    Raw4<IT> rx[QP], rd[QP], rb, x0[QP], x1[QP];  // loads under way; x of the two tiles before
    const IT* xq = x + (long long)q.t0 * ld_x + dc0 + qc;
    const IT* dq = dt + (long long)q.t0 * d.ld_dt + dc0 + qc;
    const IT* bq = bc_src + (long long)q.t0 * ld_bc + (long long)grp * N + bn;
    IT* yq = kY ? y + (long long)q.t0 * d.D + dc0 + qc : nullptr;
    auto fetch = [&](int k) {
      const int base = base_of(k);
      const long long t0 = base + qt;
      if (whole(k)) {
#pragma unroll
        for (int i = 0; i < QP; ++i)
          if (qt < kTile) {
            rx[i] = load_raw4(xq + (t0 + i * (NT / Q)) * ld_x, 4, true);
            rd[i] = load_raw4(dq + (t0 + i * (NT / Q)) * d.ld_dt, 4, true);
          }
      } else {
#pragma unroll
        for (int i = 0; i < QP; ++i) {
          const long long t = t0 + i * (NT / Q);
          const int n = t < q.len ? qn : 0;
          rx[i] = load_raw4(xq + t * ld_x, n, vec);
          rd[i] = load_raw4(dq + t * d.ld_dt, n, vec);
        }
      }
      if (has_bc) rb = load_raw4(bq + (base + bt) * ld_bc, base + bt < q.len ? 4 : 0, vec_bc);
    };
    auto form = [&](int k) {  // tile k from the registers
      const int base = base_of(k), buf = k & 1;
      const bool full = whole(k);
#pragma unroll
      for (int i = 0; i < QP; ++i) {
        const int tt = qt + i * (NT / Q);
        float xv[4], dv[4];
        rx[i].get(xv);
        rd[i].get(dv);
        if (kY) {
          x0[i] = x1[i];
          x1[i] = rx[i];
        }
        if (qt < kTile) {
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            f32x2 dl = add2(pack2(dv[c], dv[c + 1]), pack2(bias[c], bias[c + 1]));
            if (d.softplus) dl = softplus2(lo2(dl), hi2(dl), nullptr, nullptr);
            if (!full) {  // past the end the state stays as it is
              const int n = base + tt < q.len ? qn : 0;
              dl = pack2(c < n ? lo2(dl) : 0.f, c + 1 < n ? hi2(dl) : 0.f);
            }
            const f32x2 xp = pack2(xv[c], xv[c + 1]);
            sdu[buf][tt][slot((qc + c) / 2)] = Pair2{dl, MODE == kStartGrad ? xp : mul2(dl, xp)};
          }
        }
      }
      if (has_bc) {
        float v[4];
        rb.get(v);
        *reinterpret_cast<float4*>(is_c ? &sC[kY ? buf : 0][bt][bn] : &sB[buf][bt][bn]) = make_float4(v[0], v[1], v[2], v[3]);
      }
    };
    // y of tile k; xs: its x
    auto finish = [&](int k, const Raw4<IT>(&xs)[QP]) {
      if constexpr (kY) {
        const bool full = whole(k);
#pragma unroll
        for (int i = 0; i < QP; ++i) {
          const int tt = qt + i * (NT / Q);
          const long long t = k * kTile + tt;
          if (qt < kTile) {
            float xv[4], v[4];
            xs[i].get(xv);
            const float4 p = *reinterpret_cast<const float4*>(&sy[k & 1][tt][qc]);
            v[0] = fmaf(skip[0], xv[0], p.x); v[1] = fmaf(skip[1], xv[1], p.y);
            v[2] = fmaf(skip[2], xv[2], p.z); v[3] = fmaf(skip[3], xv[3], p.w);
            if (full)
              store4(yq + t * d.D, 4, true, v);
            else
              store4(yq + t * d.D, t < q.len ? qn : 0, vec, v);
          }
        }
      }
    };
    if (tiles > 0) {
      fetch(0);
      form(0);
      if (tiles > 1) fetch(1);
    }
    const int sl = slot(pr);
    for (int k = 0; k < tiles; ++k) {
      const int buf = k & 1;
      __syncthreads();
      // Two tokens at a time: a pair's loads and exponentials (which nothing in the recurrence waits
      // for) are issued a pair ahead of its recurrence.
      f32x2 e[2][2][2][2], ub[2][2][2][2];  // [turn][token][channel][two states]
      Pair2 cc[2][2];
      auto ahead = [&](int g) {
        const int w = g & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = MODE == kStartGrad ? kTile - 1 - (2 * g + i) : 2 * g + i;
          const Pair2 du = sdu[buf][t][sl];
          const Pair2 b = *reinterpret_cast<const Pair2*>(&sB[buf][t][4 * ln]);
          if (kY) cc[w][i] = *reinterpret_cast<const Pair2*>(&sC[kY ? buf : 0][t][4 * ln]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float dl = c ? hi2(du.a) : lo2(du.a), u = c ? hi2(du.b) : lo2(du.b);
            const f32x2 dd = pack2(dl, dl), uu = pack2(u, u);
            e[w][i][c][0] = ex2_2(mul2(dd, A2[c][0]));
            e[w][i][c][1] = ex2_2(mul2(dd, A2[c][1]));
            ub[w][i][c][0] = mul2(uu, b.a);
            ub[w][i][c][1] = mul2(uu, b.b);
          }
          if (!kY) dsum = add2(dsum, du.a);
        }
      };
      ahead(0);
      if (k > 0) finish(k - 1, x0);
      if (k + 1 < tiles) {
        form(k + 1);  // x0 becomes tile k's x, x1 tile k + 1's
      } else if (kY) {
#pragma unroll
        for (int i = 0; i < QP; ++i) x0[i] = x1[i];
      }
      if (k + 2 < tiles) fetch(k + 2);
      if (kY && h_saved) store_state(h_saved + (q.tile0 + k) * (long long)d.D * N, h);
      float p[8];  // [token of four][channel]
#pragma unroll
      for (int g = 0; g < kTile / 2; ++g) {
        if (g + 1 < kTile / 2) ahead(g + 1);
        const int w = g & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              h[c][j] = MODE == kStartGrad ? mul2(e[w][i][c][j], add2(ub[w][i][c][j], h[c][j]))
                                           : fma2(e[w][i][c][j], h[c][j], ub[w][i][c][j]);
            if (kY) {
              const f32x2 s = fma2(h[c][0], cc[w][i].a, mul2(h[c][1], cc[w][i].b));
              p[4 * w + 2 * i + c] = lo2(s) + hi2(s);
            }
          }
        if (kY && w == 1) {
          using Sum = LaneSums<8, NL, 1>;
          Sum::run(p, ln);
          if (Sum::holds(ln)) {
#pragma unroll
            for (int i = 0; i < Sum::KEEP; ++i) {
              const int at = Sum::index(ln) + i;
              sy[kY ? buf : 0][kY ? 2 * (g - 1) + (at >> 1) : 0][2 * pr + (at & 1)] = p[i];
            }
          }
        }
      }
    }
    __syncthreads();
    if (tiles > 0) finish(tiles - 1, x0);
    if (kY) {
      if (S_T && q.last) store_state(S_T + (long long)q.seq * d.D * N, h);
    } else {
      store_state(R + un * (long long)d.D * N, h);
      if (ln == 0) {
        if (live[0]) sum_delta[un * d.D + dch] = lo2(dsum);
        if (live[1]) sum_delta[un * d.D + dch + 1] = hi2(dsum);
      }
    }
  }
}

// Joins the segments of every sequence: cur = edge; in order (backward: reversed) of its units,
// R[u] <- cur, cur <- exp(A sum D) cur + R[u].  One thread per (sequence, channel, state); 16 units'
// loads are in flight together (57 units in turn: 14 us with 4).  The last unit contributes nothing.
__global__ void __launch_bounds__(256) ssm_join_kernel(SsmDims d, const float* __restrict__ A,
                                                       const float* __restrict__ edge, float* R,
                                                       const float* __restrict__ sum_delta, int backward) {
  constexpr int kAtOnce = 16;
  if (ssm_bad(d)) return;
  const long long DN = (long long)d.D * d.N, id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long seq = id / DN, dn = id - seq * DN;
  if (seq >= d.num_seqs) return;
  const long long u0 = d.cu ? d.unit_off[seq] : seq * d.seq_units;
  const int count = d.cu ? d.unit_off[seq + 1] - (int)u0 : d.seq_units;
  const float a2 = decay_rate(A[dn]);
  const long long ch = dn / d.N;
  float cur = edge ? edge[seq * DN + dn] : 0.f;
  for (int k = 0; k < count; k += kAtOnce) {
    float r[kAtOnce], s[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const long long u = u0 + (backward ? count - 1 - (k + i) : k + i);
      r[i] = k + i + 1 < count ? R[u * DN + dn] : 0.f;
      s[i] = k + i + 1 < count ? sum_delta[u * d.D + ch] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
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

// A lane holds four states of a channel for R rows: A, Dskip and dt_bias are read once for them and
// their states' loads are in flight together.  Bound by memory (8 bytes and 7 operations per state):
// 256 rows, D = 4096, N = 16 take 34 us with R = 1 and 29 us with R = 4 (20 us at the copy rate); few
// rows take R = 1, where threads are scarcer than loads.
template <typename IT, int NL, int R>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmDims d, int B, int num_slots, const IT* __restrict__ x,
                                                       const IT* __restrict__ dt, const float* __restrict__ A,
                                                       const IT* __restrict__ Bm, const IT* __restrict__ Cm,
                                                       const float* __restrict__ Dskip,
                                                       const float* __restrict__ dt_bias, float* __restrict__ pool,
                                                       const int32_t* __restrict__ slots, IT* __restrict__ y) {
  constexpr int N = 4 * NL;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const int ln = (int)(id % NL), ch = (int)(id / NL);
  const bool in = ch < d.D;
  const int b0 = blockIdx.y * R;
  float4 h[R];
  float xv[R], dl[R];
  float4* hp[R];
  bool live[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = b0 + r, slot = b < B ? (slots ? slots[b] : b) : -1;
    live[r] = in && slot >= 0 && slot < num_slots;
    hp[r] = reinterpret_cast<float4*>(pool + ((long long)slot * d.D + ch) * N + 4 * ln);
    h[r] = live[r] ? __ldcs(hp[r]) : make_float4(0.f, 0.f, 0.f, 0.f);
    xv[r] = live[r] ? to_f32(x[b * d.ld_x + ch]) : 0.f;
    dl[r] = live[r] ? to_f32(dt[b * d.ld_dt + ch]) : 0.f;
  }
  const float4 a = in ? *reinterpret_cast<const float4*>(A + (long long)ch * N + 4 * ln) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float bias = in && dt_bias ? dt_bias[ch] : 0.f, skip = in && Dskip ? Dskip[ch] : 0.f;
  const float a2[4] = {decay_rate(a.x), decay_rate(a.y), decay_rate(a.z), decay_rate(a.w)};
  const int g = in ? ch / d.Dg : 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = b0 + r;
    float p = 0.f;
    if (live[r]) {
      float dlt = dl[r] + bias;
      if (d.softplus) dlt = softplus_f(dlt, nullptr);
      const IT* bp = Bm + b * d.ld_b + g * N + 4 * ln;
      const IT* cp = Cm + b * d.ld_c + g * N + 4 * ln;
      const float u = dlt * xv[r];
      h[r].x = fmaf(ex2f(dlt * a2[0]), h[r].x, u * to_f32(bp[0]));
      h[r].y = fmaf(ex2f(dlt * a2[1]), h[r].y, u * to_f32(bp[1]));
      h[r].z = fmaf(ex2f(dlt * a2[2]), h[r].z, u * to_f32(bp[2]));
      h[r].w = fmaf(ex2f(dlt * a2[3]), h[r].w, u * to_f32(bp[3]));
      __stcs(hp[r], h[r]);
      p = fmaf(h[r].x, to_f32(cp[0]), fmaf(h[r].y, to_f32(cp[1]), fmaf(h[r].z, to_f32(cp[2]), h[r].w * to_f32(cp[3]))));
    }
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
    if (in && b < B && ln == 0) y[(long long)b * d.D + ch] = from_f32<IT>(live[r] ? fmaf(skip, xv[r], p) : 0.f);
  }
}

int fwd_blocks(const SsmDims& d) {
  return d.G * ((d.Dg + kFwdChannels - 1) / kFwdChannels);
}

template <typename F>
cudaError_t ssm_type(gdr_dtype dt, F f) {
  return dt == GDR_DTYPE_BF16 ? f(__nv_bfloat16{}) : f(float{});
}

unsigned unit_rows(const SsmDims& d) { return (unsigned)(d.max_units < 32768 ? d.max_units : 32768); }

}  // namespace

int ssm_vec(const SsmDims& d, size_t el, std::initializer_list<const void*> rows, std::initializer_list<const void*> bc) {
  bool v = d.Dg % 4 == 0 && d.ld_x % 4 == 0 && d.ld_dt % 4 == 0 && d.ld_dy % 4 == 0, b = d.ld_b % 4 == 0 && d.ld_c % 4 == 0;
  for (const void* p : rows) v = v && elem_ok(p, 4 * el);
  for (const void* p : bc) b = b && elem_ok(p, 4 * el);
  return (v ? 1 : 0) | (b ? 2 : 0);
}

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
  // A block takes about 80 ns a token however few there are, and an SM is full at 2.2 of them; cutting
  // sequences into segments costs the first pass (0.7 of the full one).  So segments pay below about
  // one block per SM (B = 2, T = 4096, D = 4096, N = 16, 128 blocks: 285 us against 328), and where a
  // packed batch's longest sequence, which the host does not know, may be twice the average, below
  // two.  They are made of at least 64 tokens, enough for six blocks per SM.  The rule takes a packed batch's
  // sequences for about equally long: one that outweighs the others is not cut where their number is large (D = 1024, N =
  // 16, bf16, 30000 tokens and 19 times 100: forward 2254 us, backward 5403; 20 times 1595: 225 and 719).
  const long long blocks = fwd_blocks(*d), whole = (d->T + kTile - 1) / kTile * (long long)kTile;
  d->Lseg = (int)(whole < kTile ? kTile : whole);
  if (!step && d->total > 0 && blocks * d->num_seqs < (d->cu ? 2 : 1) * kSmCount) {
    const long long want = (6ll * kSmCount + blocks - 1) / blocks;  // segments over all sequences
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
  d.vec = ssm_vec(d, el, {x, dt, y}, {Bm, Cm});
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
  const long long gx = ((long long)d.D * (d.N / 4) + 255) / 256;
  const bool four = gx * ((p->B + 3) / 4) >= 4 * kSmCount;
  const int rows = four ? 4 : 1;
  if ((p->B + rows - 1) / rows > 65535) return GDR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)((p->B + rows - 1) / rows));
  return status_of(ssm_type(p->dtype, [&](auto it) {
    using IT = decltype(it);
    return ssm_lanes(d.N, [&](auto nl) {
      constexpr int NL = decltype(nl)::value;
      const auto kernel = four ? ssm_step_kernel<IT, NL, 4> : ssm_step_kernel<IT, NL, 1>;
      kernel<<<grid, 256, 0, s>>>(d, p->B, p->num_slots, (const IT*)x, (const IT*)dt, A, (const IT*)Bm, (const IT*)Cm, Dskip,
                                  dt_bias, pool, slots, (IT*)y);
      stage_mark(s, "ssm_step");
      return cudaGetLastError();
    });
  }));
}

}  // extern "C"
