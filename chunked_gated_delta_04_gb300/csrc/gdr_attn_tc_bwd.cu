// gdr_attn_tc_bwd.cu -- attention backward on the tensor cores (include/gdr_attn.h), bf16, D up to 128.
//
//   P = e^{scale Q K^T - lse},   dS = P (dO V^T - delta),   dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K
//
// Two kernels, each of which forms P and dS anew: one takes 128 keys through the queries that see them (dK, dV), one 128 queries
// through the keys that they see (dQ).  That is seven products per pair of tiles where one kernel would do with five, but the sums stay
// in TMEM: no pass over dQ in memory for every key tile, and no atomics, whose order would change results.
// Both are persistent, one block per SM, with the same roles: a warp for the TMA copies, a thread that issues the MMAs, two
// warpgroups for the arithmetic on P and dS; thread = row of the tile in TMEM, the warpgroups take 64 columns each.
//   keys:    S^T = K Q^T and dP^T = V dO^T have the keys as rows, so that P^T and dS^T, written over them as bf16, are the
//            products' operands from TMEM.  TMEM: S^T, dP^T 128 columns each, dV, dK: all 512.  Issue order: dV, next S^T, dK, next
//            dP^T; P is formed beside dK and dP^T, dS beside dV and the next S^T.  A spare warp brings lse and delta.
//   queries: S = Q K^T and dP = dO V^T free their columns as soon as they are in registers; dS has two places of its own.
// Where the tiles are less than half of the SMs (few key heads, short sequences), the blocks of a cluster share one (Share): each
// takes every n-th step, and sums some of the rows from all blocks' shared memory, in the order of their ranks.
// Bound by the products.  B = 1, T = 8192, 32 heads on 8 of 128, causal: dK and dV 612 to 627 us, 1.75 to 1.80 PFLOP/s of the four products that
// are issued, 90 to 93 % of cuBLAS's rate; dQ 493 to 522 us, 1.58 to 1.67 PFLOP/s of its three.  2 x 4096 tokens, 16 heads of 128: 182 and 147 us
// (from the first form's 222 and 196), where beginnings and ends of items, about 5 us each, weigh more.  One key head for 8 query heads,
// T = 4096, 32 tiles of keys shared by 4 blocks each: 137 to 141 us for all three launches.
#include <algorithm>

#include "gdr_attn_tc.cuh"

namespace gdr {
namespace {

using namespace tcx;

constexpr int kThreads = 384;  // 8 warps of arithmetic, MMAs, copies, statistics, one idle
constexpr int kMmaWarp = 8, kLoadWarp = 9, kStatWarp = 10;
// Two tiles that stay, and rings of the ones that pass: three slots for what the last product of a step reads (Q, or K), two for
// what an earlier one does (dO, or V).
constexpr int kA = 3, kB = 2;

struct BwdMaps {
  CUtensorMap q, k, v, dout;
};

// Behind the tiles in shared memory.
struct BwdShared {
  float stat[2][2][kTcBlock];  // lse log2(e), delta of a query tile
  uint64_t keep_full[2], keep_empty[2], a_full[kA], a_empty[kA], b_full[kB], b_empty[kB], stat_full[2], stat_empty[2];
  uint64_t s_full, dp_full, s_free, dp_free, p_ready, ds_ready[2], done, tail_full, drain;
  uint32_t tmem_slot;
};
template <int DP>
constexpr size_t bwd_smem() { return (size_t)(2 + kA + kB) * attn_tile_bytes<DP>() + sizeof(BwdShared); }
static_assert(bwd_smem<128>() <= 227 * 1024, "shared memory of a block");

// The tiles need 1024-byte alignment; the kernels have no other shared memory.
extern __shared__ __align__(1024) unsigned char bwd_raw[];

__device__ __forceinline__ void bwd_barriers(BwdShared& b) {
  for (int i = 0; i < 2; ++i) {
    tc::mbar_init(&b.keep_full[i], 1);
    tc::mbar_init(&b.keep_empty[i], 1);
    tc::mbar_init(&b.stat_full[i], 1);
    tc::mbar_init(&b.stat_empty[i], 8);
    tc::mbar_init(&b.ds_ready[i], 8);
  }
  for (int i = 0; i < kA; ++i) {
    tc::mbar_init(&b.a_full[i], 1);
    tc::mbar_init(&b.a_empty[i], 1);
  }
  for (int i = 0; i < kB; ++i) {
    tc::mbar_init(&b.b_full[i], 1);
    tc::mbar_init(&b.b_empty[i], 1);
  }
  tc::mbar_init(&b.s_full, 1);
  tc::mbar_init(&b.dp_full, 1);
  tc::mbar_init(&b.s_free, 8);
  tc::mbar_init(&b.dp_free, 8);
  tc::mbar_init(&b.p_ready, 8);
  tc::mbar_init(&b.done, 1);
  tc::mbar_init(&b.tail_full, 1);
  tc::mbar_init(&b.drain, 1);
  tc::fence_barrier_init();
}

// The loading warp's side of a ring.
template <int DP, int N>
struct BwdLoader {
  BwdShared& b;
  unsigned char* at;
  uint64_t *full, *empty;
  uint32_t* status;
  AttnRing<N> ring;

  // The rows [r0, r0 + 128) of a head; `rows` of them are the sequence's, and with `clear` the others become zeros before the
  // tile counts as loaded.
  __device__ __forceinline__ bool load(const CUtensorMap* map, int head, long long r0, int rows, bool clear, uint32_t& tail_parity) {
    GDR_DELAY(47);
    if (!attn_warp_wait(&empty[ring.slot], ring.parity ^ 1u, status, kDevErrTimeoutBwd)) return false;
    unsigned char* const dst = at + ring.slot * attn_tile_bytes<DP>();
    const bool tail = clear && rows < kTcBlock;
    uint64_t* const bar = tail ? &b.tail_full : &full[ring.slot];
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(bar, attn_tile_bytes<DP>());
      attn_load_tile<DP>(dst, map, bar, head, r0);
    }
    if (tail) {
      const bool ok = attn_warp_wait(&b.tail_full, tail_parity, status, kDevErrTimeoutBwd);
      tail_parity ^= 1u;
      if (!ok) return false;
      attn_clear_rows<DP>(dst, rows);
      if (lane == 0) tc::mbar_arrive(&full[ring.slot]);
    }
    ring.next();
    return true;
  }
  // After a wait that ran out, the copies under way end before the block does.
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < N; ++i) {
      tc::mbar_wait(&full[ring.slot], ring.parity ^ 1u, status, kDevErrTimeoutBwd);
      ring.next();
    }
  }
};

// ------------------------------------------------------------------------------------ dK, dV
struct KeyItem {
  AttnSpan s;
  int h, j0, lo, hi;  // key head, first key, query tiles [lo, hi)
};
__device__ __forceinline__ bool key_item(const AttnDims& d, const AttnTiles& t, unsigned x, KeyItem* w) {
  int seq, tile;
  if (!attn_tile(d, t, d.Hk, x, &seq, &w->h, &tile)) return false;
  w->s = attn_span(d, seq);
  w->j0 = tile * kTcBlock;
  int lo = 0, hi = 0;
  if (w->j0 < w->s.m) attn_queries(d, w->s, w->j0, min(w->s.m, w->j0 + kTcBlock), &lo, &hi);
  w->lo = lo < hi ? lo / kTcBlock : 0;
  w->hi = lo < hi ? (hi + kTcBlock - 1) / kTcBlock : 0;
  return true;
}

template <int DP, bool Share>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkdv_tc_kernel(const __grid_constant__ BwdMaps maps, AttnDims d, AttnTiles tiles, unsigned items, AttnBwdArgs a) {
  constexpr uint32_t kTile = attn_tile_bytes<DP>();
  constexpr uint32_t kS = 0, kdP = 128, kdV = 256, kdK = 256 + DP;
  unsigned char* const keep = bwd_raw;  // K, V
  unsigned char* const a_at = keep + 2 * kTile;
  unsigned char* const b_at = a_at + kA * kTile;
  BwdShared& b = *reinterpret_cast<BwdShared*>(b_at + kB * kTile);
  const int warp = attn_warp(), lane = threadIdx.x & 31;
  uint32_t* const status = a.status;
  if (threadIdx.x == 0) bwd_barriers(b);
  if (warp == kMmaWarp) tc::tmem_alloc<512>(&b.tmem_slot);
  if (warp == kLoadWarp && lane == 0) {
    tc::tma_prefetch_desc(&maps.q);
    tc::tma_prefetch_desc(&maps.k);
    tc::tma_prefetch_desc(&maps.v);
    tc::tma_prefetch_desc(&maps.dout);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = b.tmem_slot;
  launch_wait();
  launch_next();
  const int n = Share ? attn_cluster_size() : 1, rank = Share ? (int)tc::cluster_ctarank() : 0;
  float* const part = reinterpret_cast<float*>(bwd_raw);  // Share: the block's sums, once its tiles are used up
  KeyItem w;
  bool ok = true;

  if (warp == kLoadWarp) {
    BwdLoader<DP, kA> qs{b, a_at, b.a_full, b.a_empty, status};
    BwdLoader<DP, kB> dos{b, b_at, b.b_full, b.b_empty, status};
    uint32_t kv_parity = 0, tail_parity = 0;
    for (unsigned turn = 0; ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!key_item(d, tiles, (unsigned)x, &w) || w.lo >= w.hi) continue;
      auto load_kv = [&](int which, const CUtensorMap* map) {
        ok = ok && attn_warp_wait(&b.keep_empty[which], kv_parity ^ 1u, status, kDevErrTimeoutBwd);
        if (ok && lane == 0) {
          tc::mbar_arrive_expect_tx(&b.keep_full[which], kTile);
          attn_load_tile<DP>(keep + which * kTile, map, &b.keep_full[which], w.h, w.s.k0 + w.j0);
        }
      };
      const int length = w.hi - w.lo, steps = length * d.G;
      if (rank >= steps) continue;
      load_kv(0, &maps.k);
      for (int st = rank; st < steps && ok; st += n) {
        const int g = st / length, i = w.lo + st % length;
        const long long r0 = w.s.q0 + (long long)i * kTcBlock;
        const int rows = w.s.n - i * kTcBlock;
        ok = qs.load(&maps.q, w.h * d.G + g, r0, rows, true, tail_parity);
        if (st == rank) load_kv(1, &maps.v);
        ok = ok && dos.load(&maps.dout, w.h * d.G + g, r0, rows, true, tail_parity);
      }
      kv_parity ^= 1u;
    }
    if (!ok) {
      qs.drain();
      dos.drain();
    }
  } else if (warp == kMmaWarp) {
    {
      const uint32_t leader = attn_leader();
      AttnRing<kA> qs;
      AttnRing<kB> dos;
      uint32_t kv_parity = 0, parity = 0;
      const uint32_t k_at = tc::smem_u32(keep), v_at = k_at + kTile, q_at = tc::smem_u32(a_at), do_at = tc::smem_u32(b_at);
      auto wait = [&](uint64_t* bar, uint32_t p) {
        ok = ok && attn_warp_wait(bar, p, status, kDevErrTimeoutBwd);
        tc::tc_fence_after();
        return ok;
      };
      for (unsigned turn = 0; ok; ++turn) {
        const long long x = attn_item(turn, items, n);
        if (x < 0) break;
        if (!key_item(d, tiles, (unsigned)x, &w) || w.lo >= w.hi) continue;
        const int steps = ((w.hi - w.lo) * d.G - rank + n - 1) / n;  // the block's
        if (steps <= 0) continue;
        auto scores = [&](bool last) {  // S^T of the next step
          if (!wait(&b.a_full[qs.slot], qs.parity)) return;
          attn_scores<DP>(tmem + kS, k_at, q_at + qs.slot * kTile, leader);
          attn_commit(&b.s_full, leader);
          if (last) attn_commit(&b.keep_empty[0], leader);
        };
        auto dscores = [&](bool last) {  // dP^T of the next step
          if (!wait(&b.b_full[dos.slot], dos.parity)) return;
          attn_scores<DP>(tmem + kdP, v_at, do_at + dos.slot * kTile, leader);
          attn_commit(&b.dp_full, leader);
          if (last) attn_commit(&b.keep_empty[1], leader);
        };
        if (wait(&b.keep_full[0], kv_parity)) scores(steps == 1);
        if (wait(&b.keep_full[1], kv_parity)) dscores(steps == 1);
        kv_parity ^= 1u;
        for (int it = 0; it < steps && ok; ++it) {
          const int q_slot = qs.slot, do_slot = dos.slot;
          const bool more = it + 1 < steps, last = it + 2 == steps;
          qs.next();
          dos.next();
          GDR_DELAY(45);
          if (!wait(&b.p_ready, parity)) break;
          attn_product<DP, 64>(tmem + kdV, tmem + kS, do_at + do_slot * kTile, it > 0, leader);
          attn_commit(&b.b_empty[do_slot], leader);
          if (more) scores(last);
          GDR_DELAY(46);
          if (!wait(&b.ds_ready[0], parity)) break;
          attn_product<DP, 64>(tmem + kdK, tmem + kdP, q_at + q_slot * kTile, it > 0, leader);
          attn_commit(&b.a_empty[q_slot], leader);
          if (more)
            dscores(last);
          else
            attn_commit(&b.done, leader);
          parity ^= 1u;
        }
      }
      if (!ok) {  // the products under way end before their memory is given back
        attn_commit(&b.drain, leader);
        attn_warp_wait(&b.drain, 0, status, kDevErrTimeoutBwd);
      }
    }
    __syncwarp();
  } else if (warp == kStatWarp) {
    AttnRing<2> ring;
    for (unsigned turn = 0; ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!key_item(d, tiles, (unsigned)x, &w) || w.lo >= w.hi) continue;
      const int length = w.hi - w.lo, steps = length * d.G;
      for (int st = rank; st < steps; st += n) {
        const int g = st / length, i = w.lo + st % length;
        const long long at = w.s.lse0 + (long long)(w.h * d.G + g) * d.Tq;
        float ls[4], dl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = i * kTcBlock + 32 * e + lane;
          const bool on = r < w.s.n;
          ls[e] = on ? a.lse[at + r] * kLog2e : INFINITY;
          dl[e] = on ? a.delta[at + r] : 0.f;
          if (ls[e] == -INFINITY) ls[e] = INFINITY;  // a query that sees nothing: e^-infinity
        }
        ok = attn_warp_wait(&b.stat_empty[ring.slot], ring.parity ^ 1u, status, kDevErrTimeoutBwd);
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          b.stat[ring.slot][0][32 * e + lane] = ls[e];
          b.stat[ring.slot][1][32 * e + lane] = dl[e];
        }
        __syncwarp();
        GDR_DELAY_WARP(57);
        if (lane == 0) tc::mbar_arrive(&b.stat_full[ring.slot]);
        ring.next();
      }
    }
  } else if (warp < 8) {
    const int half = warp >> 2, row = threadIdx.x & 127, col = 64 * half;
    const uint32_t s_col = tc::tmem_lane_addr(tmem, warp, kS + col), dp_col = tc::tmem_lane_addr(tmem, warp, kdP + col);
    const float c = d.scale * kLog2e;
    uint32_t parity = 0, done_parity = 0;
    AttnRing<2> ring;
    for (unsigned turn = 0; ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!key_item(d, tiles, (unsigned)x, &w)) continue;
      const int j = w.j0 + row, off = w.s.m - w.s.n;
      // the queries [from, to) that see this key; tiles [.., ..) in which every query sees every key of the tile
      const int from = d.causal ? j - off : 0;
      const long long to = d.window ? (long long)j - off + d.window : w.s.n;
      const int j_last = w.j0 + kTcBlock - 1;
      const int whole_from = d.causal ? j_last - off : 0;
      const long long whole_to = d.window ? (long long)w.j0 - off + d.window : (1ll << 40);
      const int length = w.hi - w.lo, steps = length * d.G;
      for (int st = rank; st < steps; st += n) {
        const int i = w.lo + (d.G == 1 ? st : st % length);
        ok = attn_warp_wait(&b.stat_full[ring.slot], ring.parity, status, kDevErrTimeoutBwd);
        ok = ok && attn_warp_wait(&b.s_full, parity, status, kDevErrTimeoutBwd);
        if (!ok) break;
        tc::tc_fence_after();
        const int i0 = i * kTcBlock;
        float p[64], dp[64];
        tc::tmem_ld32(s_col, p);
        tc::tmem_ld32(s_col + 32, p + 32);
        tc::tmem_wait_ld();
        const float* ls = b.stat[ring.slot][0] + col;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(ls + e);
          p[e] = ex2f(fmaf(p[e], c, -l4.x));
          p[e + 1] = ex2f(fmaf(p[e + 1], c, -l4.y));
          p[e + 2] = ex2f(fmaf(p[e + 2], c, -l4.z));
          p[e + 3] = ex2f(fmaf(p[e + 3], c, -l4.w));
        }
        if (i0 < whole_from || i0 + kTcBlock > whole_to) {
          const int a0 = from - i0 - col;
          const int a1 = (int)min(to - i0 - col, 1ll << 20);
#pragma unroll
          for (int e = 0; e < 64; ++e) p[e] = e >= a0 && e < a1 ? p[e] : 0.f;
        }
        attn_put64(s_col, p);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        GDR_DELAY(41);
        if (lane == 0) tc::mbar_arrive(&b.p_ready);
        ok = attn_warp_wait(&b.dp_full, parity, status, kDevErrTimeoutBwd);
        if (!ok) break;
        tc::tc_fence_after();
        tc::tmem_ld32(dp_col, dp);
        tc::tmem_ld32(dp_col + 32, dp + 32);
        tc::tmem_wait_ld();
        const float* dl = b.stat[ring.slot][1] + col;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 d4 = *reinterpret_cast<const float4*>(dl + e);
          dp[e] = p[e] * (dp[e] - d4.x);
          dp[e + 1] = p[e + 1] * (dp[e + 1] - d4.y);
          dp[e + 2] = p[e + 2] * (dp[e + 2] - d4.z);
          dp[e + 3] = p[e + 3] * (dp[e + 3] - d4.w);
        }
        attn_put64(dp_col, dp);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        GDR_DELAY(42);
        if (lane == 0) {
          tc::mbar_arrive(&b.ds_ready[0]);
          tc::mbar_arrive(&b.stat_empty[ring.slot]);
        }
        parity ^= 1u;
        ring.next();
      }
      if (!ok) break;
      const bool any = rank < steps;
      if (any) {
        ok = attn_warp_wait(&b.done, done_parity, status, kDevErrTimeoutBwd);
        done_parity ^= 1u;
        if (!ok) break;
        tc::tc_fence_after();
      }
      // the first warpgroup stores dV, the second dK
      const uint32_t from_t = tc::tmem_lane_addr(tmem, warp, half ? kdK : kdV);
      if constexpr (Share) {
        put_part<DP, DP>(part + half * kTcBlock * DP, row, 0, from_t, half ? d.scale : 1.f, any);
      } else {
        __nv_bfloat16* const out = (__nv_bfloat16*)(half ? a.dk : a.dv) + ((w.s.k0 + j) * d.Hk + w.h) * (long long)d.D;
        attn_store_row<DP>(from_t, out, d.D, half ? d.scale : 1.f, any, j < w.s.m);
      }
      tc::tc_fence_before();  // read before the next item's first product into them, which the next arrival allows
    }
  }
  if constexpr (Share) {
    __syncwarp();
    GDR_DELAY_WARP(62);
    tc::cluster_sync();
    const long long x = attn_item(0, items, n);
    if (warp < 8 && x >= 0 && key_item(d, tiles, (unsigned)x, &w)) {
      const long long at = ((w.s.k0 + w.j0) * d.Hk + w.h) * (long long)d.D, ld = (long long)d.Hk * d.D;
      sum_parts<DP>(part, rank, n, (__nv_bfloat16*)a.dv + at, ld, w.s.m - w.j0, d.D, 1.f);
      sum_parts<DP>(part + kTcBlock * DP, rank, n, (__nv_bfloat16*)a.dk + at, ld, w.s.m - w.j0, d.D, 1.f);
    }
    __syncwarp();
    tc::cluster_sync();  // no block ends while others read it
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------- dQ
struct QueryItem {
  AttnSpan s;
  int h, i0, lo, hi;  // query head, first query, key tiles [lo, hi)
};
__device__ __forceinline__ bool query_item(const AttnDims& d, const AttnTiles& t, unsigned x, QueryItem* w) {
  int seq, tile;
  if (!attn_tile(d, t, d.Hq, x, &seq, &w->h, &tile)) return false;
  w->s = attn_span(d, seq);
  w->i0 = tile * kTcBlock;
  int lo = 0, hi = 0;
  if (w->i0 < w->s.n) attn_keys(d, w->s, w->i0, min(w->s.n, w->i0 + kTcBlock), &lo, &hi);
  w->lo = lo < hi ? lo / kTcBlock : 0;
  w->hi = lo < hi ? (hi + kTcBlock - 1) / kTcBlock : 0;
  return true;
}

template <int DP, bool Share>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_tc_kernel(const __grid_constant__ BwdMaps maps, AttnDims d, AttnTiles tiles, unsigned items, AttnBwdArgs a) {
  constexpr uint32_t kTile = attn_tile_bytes<DP>();
  constexpr uint32_t kS = 0, kdP = 128, kdQ = 256, kdS = 384;  // dS: two places of 64 columns
  unsigned char* const keep = bwd_raw;  // Q, dO
  unsigned char* const a_at = keep + 2 * kTile;
  unsigned char* const b_at = a_at + kA * kTile;
  BwdShared& b = *reinterpret_cast<BwdShared*>(b_at + kB * kTile);
  const int warp = attn_warp(), lane = threadIdx.x & 31;
  uint32_t* const status = a.status;
  if (threadIdx.x == 0) bwd_barriers(b);
  if (warp == kMmaWarp) tc::tmem_alloc<512>(&b.tmem_slot);
  if (warp == kLoadWarp && lane == 0) {
    tc::tma_prefetch_desc(&maps.q);
    tc::tma_prefetch_desc(&maps.k);
    tc::tma_prefetch_desc(&maps.v);
    tc::tma_prefetch_desc(&maps.dout);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = b.tmem_slot;
  launch_wait();
  launch_next();
  const int n = Share ? attn_cluster_size() : 1, rank = Share ? (int)tc::cluster_ctarank() : 0;
  float* const part = reinterpret_cast<float*>(bwd_raw);  // Share: the block's sums, once its tiles are used up
  QueryItem w;
  bool ok = true;

  if (warp == kLoadWarp) {
    BwdLoader<DP, kA> ks{b, a_at, b.a_full, b.a_empty, status};
    BwdLoader<DP, kB> vs{b, b_at, b.b_full, b.b_empty, status};
    uint32_t q_parity = 0, tail_parity = 0;
    for (unsigned turn = 0; ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!query_item(d, tiles, (unsigned)x, &w) || w.lo >= w.hi) continue;
      auto load_q = [&](int which, const CUtensorMap* map) {
        ok = ok && attn_warp_wait(&b.keep_empty[which], q_parity ^ 1u, status, kDevErrTimeoutBwd);
        if (ok && lane == 0) {
          tc::mbar_arrive_expect_tx(&b.keep_full[which], kTile);
          attn_load_tile<DP>(keep + which * kTile, map, &b.keep_full[which], w.h, w.s.q0 + w.i0);
        }
      };
      if (w.lo + rank >= w.hi) continue;
      load_q(0, &maps.q);
      for (int j = w.lo + rank; j < w.hi && ok; j += n) {
        const long long r0 = w.s.k0 + (long long)j * kTcBlock;
        const int rows = w.s.m - j * kTcBlock;
        ok = ks.load(&maps.k, w.h / d.G, r0, rows, true, tail_parity);
        if (j == w.lo + rank) load_q(1, &maps.dout);
        ok = ok && vs.load(&maps.v, w.h / d.G, r0, rows, false, tail_parity);  // values are not summed here
      }
      q_parity ^= 1u;
    }
    if (!ok) {
      ks.drain();
      vs.drain();
    }
  } else if (warp == kMmaWarp) {
    {
      const uint32_t leader = attn_leader();
      AttnRing<kA> ks;
      AttnRing<kB> vs;
      AttnRing<2> place;  // of dS
      uint32_t q_parity = 0, free_parity = 1;  // s_free, dp_free: of the step before
      const uint32_t q_at = tc::smem_u32(keep), do_at = q_at + kTile, k_at = tc::smem_u32(a_at), v_at = tc::smem_u32(b_at);
      auto wait = [&](uint64_t* bar, uint32_t p) {
        ok = ok && attn_warp_wait(bar, p, status, kDevErrTimeoutBwd);
        tc::tc_fence_after();
        return ok;
      };
      for (unsigned turn = 0; ok; ++turn) {
        const long long x = attn_item(turn, items, n);
        if (x < 0) break;
        if (!query_item(d, tiles, (unsigned)x, &w) || w.lo >= w.hi) continue;
        const int steps = (w.hi - w.lo - rank + n - 1) / n;  // the block's
        if (steps <= 0) continue;
        auto scores = [&](int it) {  // S and dP of a step
          if (it == 0) wait(&b.keep_full[0], q_parity);
          wait(&b.a_full[ks.slot], ks.parity);
          if (!wait(&b.s_free, free_parity)) return;
          attn_scores<DP>(tmem + kS, q_at, k_at + ks.slot * kTile, leader);
          attn_commit(&b.s_full, leader);
          if (it + 1 == steps) attn_commit(&b.keep_empty[0], leader);
          if (it == 0) wait(&b.keep_full[1], q_parity);
          wait(&b.b_full[vs.slot], vs.parity);
          if (!wait(&b.dp_free, free_parity)) return;
          attn_scores<DP>(tmem + kdP, do_at, v_at + vs.slot * kTile, leader);
          attn_commit(&b.dp_full, leader);
          attn_commit(&b.b_empty[vs.slot], leader);
          if (it + 1 == steps) attn_commit(&b.keep_empty[1], leader);
          free_parity ^= 1u;
          ks.next();
          vs.next();
        };
        int k_slot = ks.slot;
        scores(0);
        q_parity ^= 1u;
        for (int it = 0; it < steps && ok; ++it) {
          const int next_slot = ks.slot;
          if (it + 1 < steps) scores(it + 1);
          // (a barrier for each place: the step after this one may be through before this wait begins)
          GDR_DELAY(44);
          if (!wait(&b.ds_ready[place.slot], place.parity)) break;
          attn_product<DP>(tmem + kdQ, tmem + kdS + 64 * place.slot, k_at + k_slot * kTile, it > 0, leader);
          attn_commit(&b.a_empty[k_slot], leader);
          if (it + 1 == steps) attn_commit(&b.done, leader);
          k_slot = next_slot;
          place.next();
        }
      }
      if (!ok) {  // the products under way end before their memory is given back
        attn_commit(&b.drain, leader);
        attn_warp_wait(&b.drain, 0, status, kDevErrTimeoutBwd);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    const int half = warp >> 2, row = threadIdx.x & 127, col = 64 * half;
    const uint32_t s_col = tc::tmem_lane_addr(tmem, warp, kS + col), dp_col = tc::tmem_lane_addr(tmem, warp, kdP + col);
    const uint32_t ds_col = tc::tmem_lane_addr(tmem, warp, kdS + 32 * half);
    const float c = d.scale * kLog2e;
    uint32_t parity = 0, done_parity = 0, place = 0;
    for (unsigned turn = 0; ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!query_item(d, tiles, (unsigned)x, &w)) continue;
      const int i = w.i0 + row, off = w.s.m - w.s.n;
      const bool mine = i < w.s.n;
      const long long at = w.s.lse0 + (long long)w.h * d.Tq + i;
      float ls = mine ? a.lse[at] * kLog2e : INFINITY;
      if (ls == -INFINITY) ls = INFINITY;  // a query that sees nothing: e^-infinity
      const float dl = mine ? a.delta[at] : 0.f;
      const int from = d.window ? max(0, i + off - d.window + 1) : 0, to = d.causal ? min(w.s.m, i + off + 1) : w.s.m;
      const int i_last = w.i0 + kTcBlock - 1;
      const int whole_to = d.causal ? min(w.s.m, w.i0 + off + 1) : w.s.m, whole_from = d.window ? i_last + off - d.window + 1 : 0;
      for (int j = w.lo + rank; j < w.hi; j += n) {
        ok = attn_warp_wait(&b.s_full, parity, status, kDevErrTimeoutBwd);
        if (!ok) break;
        tc::tc_fence_after();
        float p[64], dp[64];
        tc::tmem_ld32(s_col, p);
        tc::tmem_ld32(s_col + 32, p + 32);
        tc::tmem_wait_ld();
        tc::tc_fence_before();
        __syncwarp();
        GDR_DELAY_WARP(58);
        if (lane == 0) tc::mbar_arrive(&b.s_free);
#pragma unroll
        for (int e = 0; e < 64; ++e) p[e] = ex2f(fmaf(p[e], c, -ls));
        const int j0 = j * kTcBlock;
        const bool partial = j0 + kTcBlock > whole_to || j0 < whole_from;
        ok = attn_warp_wait(&b.dp_full, parity, status, kDevErrTimeoutBwd);
        if (!ok) break;
        tc::tc_fence_after();
        tc::tmem_ld32(dp_col, dp);
        tc::tmem_ld32(dp_col + 32, dp + 32);
        tc::tmem_wait_ld();
        tc::tc_fence_before();
        __syncwarp();
        GDR_DELAY_WARP(59);
        if (lane == 0) tc::mbar_arrive(&b.dp_free);
#pragma unroll
        for (int e = 0; e < 64; ++e) dp[e] = p[e] * (dp[e] - dl);
        if (partial) {
          const int a0 = from - j0 - col, a1 = to - j0 - col;
#pragma unroll
          for (int e = 0; e < 64; ++e) dp[e] = e >= a0 && e < a1 ? dp[e] : 0.f;
        }
        attn_put64(ds_col + 64 * place, dp);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        GDR_DELAY(43);
        if (lane == 0) tc::mbar_arrive(&b.ds_ready[place]);
        parity ^= 1u;
        place ^= 1u;
      }
      if (!ok) break;
      const bool any = w.lo + rank < w.hi;
      if (any) {
        ok = attn_warp_wait(&b.done, done_parity, status, kDevErrTimeoutBwd);
        done_parity ^= 1u;
        if (!ok) break;
        tc::tc_fence_after();
      }
      // each warpgroup stores half of the features
      const uint32_t from_t = tc::tmem_lane_addr(tmem, warp, kdQ + half * (DP / 2));
      if constexpr (Share) {
        put_part<DP, DP / 2>(part, row, half * (DP / 2), from_t, d.scale, any);
      } else {
        __nv_bfloat16* const out = (__nv_bfloat16*)a.dq + ((w.s.q0 + i) * d.Hq + w.h) * (long long)d.D + half * (DP / 2);
        attn_store_row<DP / 2>(from_t, out, d.D - half * (DP / 2), d.scale, any, mine);
      }
      tc::tc_fence_before();  // read before the next item's first product into it, which the next arrival allows
    }
  }
  if constexpr (Share) {
    __syncwarp();
    GDR_DELAY_WARP(62);
    tc::cluster_sync();
    const long long x = attn_item(0, items, n);
    if (warp < 8 && x >= 0 && query_item(d, tiles, (unsigned)x, &w)) {
      const long long at = ((w.s.q0 + w.i0) * d.Hq + w.h) * (long long)d.D, ld = (long long)d.Hq * d.D;
      sum_parts<DP>(part, rank, n, (__nv_bfloat16*)a.dq + at, ld, w.s.n - w.i0, d.D, 1.f);
    }
    __syncwarp();
    tc::cluster_sync();  // no block ends while others read it
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t bwd(const AttnDims& d, const AttnTiles& tq, const AttnTiles& tk, const AttnBwdArgs& a, cudaStream_t s) {
  BwdMaps maps;
  const long long rows_q = (long long)d.B * d.Tq, rows_k = (long long)d.B * d.Tk;
  if (!attn_map(&maps.q, a.q, d.D, d.Hq, rows_q, d.ld_q) || !attn_map(&maps.k, a.k, d.D, d.Hk, rows_k, d.ld_k) ||
      !attn_map(&maps.v, a.v, d.D, d.Hk, rows_k, d.ld_v) || !attn_map(&maps.dout, a.dout, d.D, d.Hq, rows_q, d.ld_do))
    return cudaErrorInvalidValue;
  auto go = [&](auto kernel, auto shared, long long items, long long steps, const AttnTiles& t, const char* stage) {
    constexpr size_t smem = bwd_smem<DP>();
    const int n = attn_sharers(items, steps);
    cudaError_t e = set_smem_once(n > 1 ? (const void*)shared : (const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    e = n > 1 ? attn_launch(shared, items * n, kThreads, smem, n, s, maps, d, t, (unsigned)items, a)
              : attn_launch(kernel, std::min<long long>(items, kSmCount), kThreads, smem, 1, s, maps, d, t, (unsigned)items, a);
    if (e != cudaSuccess) return e;
    stage_mark(s, stage);
    return cudaGetLastError();
  };
  const cudaError_t e = go(attn_dkdv_tc_kernel<DP, false>, attn_dkdv_tc_kernel<DP, true>, attn_tile_count(d, true, kTcBlock) * d.Hk,
                           (long long)((d.Tq + kTcBlock - 1) / kTcBlock) * d.G, tk, "attn_dkdv");
  if (e != cudaSuccess) return e;
  return go(attn_dq_tc_kernel<DP, false>, attn_dq_tc_kernel<DP, true>, attn_tile_count(d, false, kTcBlock) * d.Hq,
            (d.Tk + kTcBlock - 1) / kTcBlock, tq, "attn_dq");
}

}  // namespace

cudaError_t launch_attn_bwd_tc(const AttnDims& d, const AttnTiles& tq, const AttnTiles& tk, const AttnBwdArgs& a, cudaStream_t s) {
  return d.D > 64 ? bwd<128>(d, tq, tk, a, s) : bwd<64>(d, tq, tk, a, s);
}

}  // namespace gdr
