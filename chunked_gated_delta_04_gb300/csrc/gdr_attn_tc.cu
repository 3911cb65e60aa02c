// gdr_attn_tc.cu -- attention forward on the tensor cores (include/gdr_attn.h), bf16, D up to 128.
//
//   S = Q K^T,   P = e^{scale S - scale m},   O += P V,   o = O / l,   lse = scale m + log l
//
// per query with m the running maximum of its scores and l the running sum of e^..  A block takes two lanes of work through the
// visible keys, 128 at a time, so that the tensor core works on one while the other's scores are exponentiated, and goes on to its
// next item (persistent, one block per SM).  The lanes are two tiles of 128 queries of a head, or, where that leaves SMs without
// work (Split), the even and the odd key blocks of one tile, which are joined at the end; where even these tiles are less than half
// of the SMs, the blocks of a cluster take two of its lanes each, and are joined through shared memory.  Roles:
//   warp 9     loads Q, then K and V tiles by TMA into a ring of slots
//   warp 8     issues the MMAs: S_t = Q_t K_j^T (both operands in shared memory), O_t += P_t V_j (P_t from TMEM)
//   warps 4 t  the softmax of lane t, a thread per query: S from TMEM to registers, P as bf16 to TMEM over S
// In TMEM: S_t (128 columns, P_t in its first 64) and O_t (DP columns).  Issue order: O_0, next S_0, O_1, next S_1, so that
// each lane's softmax runs beside the other lane's two products; MMAs of a block are executed in order, which makes
// S's place free for the next scores once P V is issued.
// The maximum that P is formed against (m) follows the true one only when that has grown by more than 2^8: then O and
// l are rescaled; else P is up to 2^8, which bf16 holds as exactly as 1.
// B = 1, T = 8192, 32 heads on 8 of 128, causal: 319 to 338 us, 1.63 to 1.72 PFLOP/s of the formula's operations, 84 to 89 % of cuBLAS's rate; a pair
// of tiles takes 2630 cycles, its products alone 2048: what is left is the wait of each lane's products for its softmax (1370
// cycles, 780 of them exponentials and sums).  Split: three parts of 515 queries, 8 heads of 64, a window of 1024: 12.4 to 13.4 us, 2 more with one lane.
#include <algorithm>

#include "gdr_attn_tc.cuh"

namespace gdr {
namespace {

using namespace tcx;

constexpr int NT = 2;  // lanes of work
template <int DP, bool Split>
struct FwdShape {
  static constexpr int kThreads = 384;  // registers move between whole warpgroups
  static constexpr uint32_t kTile = attn_tile_bytes<DP>();
  static constexpr int kQ = Split ? 1 : 2;          // tiles of queries
  static constexpr int kSlots = DP == 128 ? 4 : 6;  // of the ring of K and V tiles
  static constexpr size_t kSmem = 1024 + (size_t)(kQ + kSlots) * kTile;
  static constexpr uint32_t kO = NT * 128;  // first column of O_0
};

struct FwdMaps {
  CUtensorMap q, k, v;
};

// An item: a head's queries i0 .. of a sequence, and the key blocks [lo, hi) of each tile (none: both 0) and of all.
struct FwdItem {
  AttnSpan s;
  int h, i0, lo[NT], hi[NT], first, last;
};

template <int Q>
__device__ __forceinline__ bool fwd_item(const AttnDims& d, const AttnTiles& t, unsigned x, FwdItem* w) {
  int seq, tile;
  if (!attn_tile(d, t, d.Hq, x, &seq, &w->h, &tile)) return false;
  w->s = attn_span(d, seq);
  w->i0 = tile * Q * kTcBlock;
  w->first = 1 << 30;
  w->last = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int a = w->i0 + i * kTcBlock;
    int lo = 0, hi = 0;
    if (i < Q && a < w->s.n) attn_keys(d, w->s, a, min(w->s.n, a + kTcBlock), &lo, &hi);
    const bool any = lo < hi;
    w->lo[i] = any ? lo / kTcBlock : 0;
    w->hi[i] = any ? (hi + kTcBlock - 1) / kTcBlock : 0;
    if (any) {
      w->first = min(w->first, w->lo[i]);
      w->last = max(w->last, w->hi[i]);
    }
  }
  return true;
}

// Split, and Share: the blocks of a cluster on one tile.
template <int DP, bool Split, bool Share>
__global__ void __launch_bounds__(FwdShape<DP, Split>::kThreads, 1)
    attn_fwd_tc_kernel(const __grid_constant__ FwdMaps maps, AttnDims d, AttnTiles tiles, unsigned items, AttnFwdArgs a) {
  using Shape = FwdShape<DP, Split>;
  constexpr int ST = Shape::kSlots, Q = Shape::kQ;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t q_full[NT], q_empty[NT], kv_full[ST], kv_empty[ST], s_full[NT], p_half[NT], p_ready[NT], o_done[NT], tail_full, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ float joint[Split ? 2 : 1][2][NT][kTcBlock];  // Split: maxima and sums of an item's two lanes, of the next item's
  const int n = Share ? attn_cluster_size() : 1, rank = Share ? (int)tc::cluster_ctarank() : 0;
  // Split: the block's key blocks of an item are the first + own(i)-th ones, lane i & 1
  auto own = [&](int i) { return (i >> 1) * 2 * n + 2 * rank + (i & 1); };
  auto own_count = [&](int all) { return all <= 0 ? 0 : all / (2 * n) * 2 + max(0, min(2, all % (2 * n) - 2 * rank)); };
  float* const part = reinterpret_cast<float*>(align1024(raw));  // shared items: the block's O, once its tiles are used up
  unsigned char* const sq = align1024(raw);
  unsigned char* const skv = sq + Q * Shape::kTile;
  const int warp = attn_warp(), lane = threadIdx.x & 31;
  uint32_t* const status = a.status;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NT; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&p_half[i], 4);
      tc::mbar_init(&p_ready[i], 4);
      tc::mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&kv_full[i], 1);
      tc::mbar_init(&kv_empty[i], 1);
    }
    tc::mbar_init(&tail_full, 1);
    tc::mbar_init(&drain, 1);
    tc::fence_barrier_init();
  }
  if (warp == 4 * NT) tc::tmem_alloc<512>(&tmem_slot);
  if (warp == 4 * NT + 1 && lane == 0) {
    tc::tma_prefetch_desc(&maps.q);
    tc::tma_prefetch_desc(&maps.k);
    tc::tma_prefetch_desc(&maps.v);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  launch_wait();
  launch_next();
  if (blockIdx.x == 0 && threadIdx.x == 0 && !d.cu_q) *status = 0;  // of a packed batch: the tile table's kernel

  // Registers: three warpgroups are launched with 168 a thread; 2 x 216 + 72 is the same sum.
  // (Each count stands in its role's own branch: the compiler allots the code behind it by it.)
  if (warp >= 4 * NT) {
    regs_less<72>();
    if (warp == 4 * NT + 1) {
    // ------------------------------------------------------------------------------- loads
    AttnRing<ST> ring;
    uint32_t q_parity = 0, tail_parity = 0;
    bool ok = true;
    auto load_kv = [&](const CUtensorMap* map, const FwdItem& w, int j, bool value) {
      GDR_DELAY(49);
      ok = ok && attn_warp_wait(&kv_empty[ring.slot], ring.parity ^ 1u, status, kDevErrTimeoutFwd);
      if (!ok) return;
      unsigned char* const dst = skv + ring.slot * Shape::kTile;
      const int rows = w.s.m - j * kTcBlock;  // of the sequence in this tile
      // The values behind a sequence's end: a warp clears them before the tile counts as loaded.
      uint64_t* const bar = value && rows < kTcBlock ? &tail_full : &kv_full[ring.slot];
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bar, Shape::kTile);
        attn_load_tile<DP>(dst, map, bar, w.h / d.G, w.s.k0 + (long long)j * kTcBlock);
      }
      if (bar == &tail_full) {
        ok = attn_warp_wait(&tail_full, tail_parity, status, kDevErrTimeoutFwd);
        tail_parity ^= 1u;
        if (!ok) return;
        attn_clear_rows<DP>(dst, rows);
        if (lane == 0) tc::mbar_arrive(&kv_full[ring.slot]);
      }
      ring.next();
    };
    FwdItem w;
    for (unsigned turn = 0; ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!fwd_item<Q>(d, tiles, (unsigned)x, &w)) continue;
      auto load_q = [&](int i) {
        ok = ok && attn_warp_wait(&q_empty[i], (q_parity >> i & 1u) ^ 1u, status, kDevErrTimeoutFwd);
        if (ok && lane == 0) {
          tc::mbar_arrive_expect_tx(&q_full[i], Shape::kTile);
          attn_load_tile<DP>(sq + i * Shape::kTile, &maps.q, &q_full[i], w.h, w.s.q0 + w.i0 + i * kTcBlock);
        }
        q_parity ^= 1u << i;
      };
      if (w.first >= w.last) continue;
      if constexpr (Split) {  // the order in which they are used: two blocks of scores are ahead of the values
        const int count = own_count(w.last - w.first);
        if (count == 0) continue;
        load_q(0);
        load_kv(&maps.k, w, w.first + own(0), false);
        if (count > 1) load_kv(&maps.k, w, w.first + own(1), false);
        for (int i = 0; i < count && ok; ++i) {
          load_kv(&maps.v, w, w.first + own(i), true);
          if (i + 2 < count) load_kv(&maps.k, w, w.first + own(i + 2), false);
        }
      } else {
        if (w.hi[0]) load_q(0);
        load_kv(&maps.k, w, w.first, false);
        if (w.hi[1]) load_q(1);
        for (int j = w.first; j < w.last && ok; ++j) {
          if (j > w.first) load_kv(&maps.k, w, j, false);
          load_kv(&maps.v, w, j, true);
        }
      }
    }
    // after a wait that ran out, the copies under way end before the block does
    if (!ok)
      for (int i = 0; i < ST; ++i) {
        tc::mbar_wait(&kv_full[ring.slot], ring.parity ^ 1u, status, kDevErrTimeoutFwd);
        ring.next();
      }
    } else if (warp == 4 * NT) {
    // -------------------------------------------------------------------------------- MMAs
    {
      const uint32_t leader = attn_leader();
      AttnRing<ST> ring;
      uint32_t q_parity = 0, p_parity = 0;
      const uint32_t q_at = tc::smem_u32(sq), kv_at = tc::smem_u32(skv);
      bool ok = true;
      FwdItem w;
      for (unsigned turn = 0; ok; ++turn) {
        const long long x = attn_item(turn, items, n);
        if (x < 0) break;
        if (!fwd_item<Q>(d, tiles, (unsigned)x, &w)) continue;
        auto value_product = [&](int i, int slot, bool more) {  // O_i (+)= P_i V, the first half of it once that half of P is there
          const uint32_t o = tmem + Shape::kO + i * DP, p = tmem + i * 128, v = kv_at + slot * Shape::kTile, parity = p_parity >> i & 1u;
          p_parity ^= 1u << i;
          ok = ok && attn_warp_wait(&p_half[i], parity, status, kDevErrTimeoutFwd);
          if (!ok) return false;
          tc::tc_fence_after();
          attn_product<DP, 32, 0, 4>(o, p, v, more, leader);
          ok = attn_warp_wait(&p_ready[i], parity, status, kDevErrTimeoutFwd);
          if (!ok) return false;
          tc::tc_fence_after();
          attn_product<DP, 32, 4, 8>(o, p, v, true, leader);
          return true;
        };
        auto scores = [&](int i, int slot, int j) {  // S_i of key block j
          attn_scores<DP>(tmem + i * 128, q_at + i * Shape::kTile, kv_at + slot * Shape::kTile, leader);
          attn_commit(&s_full[i], leader);
          if (j + 1 == w.hi[i]) attn_commit(&q_empty[i], leader);
        };
        if constexpr (Split) {
          const int count = w.first < w.last ? own_count(w.last - w.first) : 0;
          if (count == 0) continue;
          auto next_scores = [&](int i) {
            ok = ok && attn_warp_wait(&kv_full[ring.slot], ring.parity, status, kDevErrTimeoutFwd);
            if (!ok) return;
            tc::tc_fence_after();
            attn_scores<DP>(tmem + (i & 1) * 128, q_at, kv_at + ring.slot * Shape::kTile, leader);
            attn_commit(&s_full[i & 1], leader);
            if (i + 1 == count) attn_commit(&q_empty[0], leader);
            attn_commit(&kv_empty[ring.slot], leader);
            ring.next();
          };
          ok = attn_warp_wait(&q_full[0], q_parity & 1u, status, kDevErrTimeoutFwd);
          q_parity ^= 1u;
          next_scores(0);
          if (count > 1) next_scores(1);
          for (int j = 0; j < count && ok; ++j) {
            const int i = j & 1;
            ok = attn_warp_wait(&kv_full[ring.slot], ring.parity, status, kDevErrTimeoutFwd);
            GDR_DELAY(48);
            if (!value_product(i, ring.slot, j > 1)) break;
            attn_commit(&o_done[i], leader);
            attn_commit(&kv_empty[ring.slot], leader);
            ring.next();
            if (j + 2 < count) next_scores(j + 2);
          }
          continue;
        }
        if (w.first < w.last) {
          ok = attn_warp_wait(&kv_full[ring.slot], ring.parity, status, kDevErrTimeoutFwd);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (w.hi[i] == 0) continue;
            ok = ok && attn_warp_wait(&q_full[i], q_parity >> i & 1u, status, kDevErrTimeoutFwd);
            q_parity ^= 1u << i;
            tc::tc_fence_after();
            if (ok && w.lo[i] == w.first) scores(i, ring.slot, w.first);
          }
          attn_commit(&kv_empty[ring.slot], leader);
          ring.next();
        }
        for (int j = w.first; j < w.last && ok; ++j) {
          const int v_slot = ring.slot;
          ok = attn_warp_wait(&kv_full[v_slot], ring.parity, status, kDevErrTimeoutFwd);
          ring.next();
          bool k_here = false;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (!ok) break;
            if (j >= w.lo[i] && j < w.hi[i]) {
              GDR_DELAY(48);
              if (!value_product(i, v_slot, j > w.lo[i])) break;
              attn_commit(&o_done[i], leader);
            }
            if (j + 1 >= w.lo[i] && j + 1 < w.hi[i]) {
              if (!k_here) {
                ok = attn_warp_wait(&kv_full[ring.slot], ring.parity, status, kDevErrTimeoutFwd);
                if (!ok) break;
                k_here = true;
              }
              tc::tc_fence_after();
              scores(i, ring.slot, j + 1);
            }
          }
          if (!ok) break;
          attn_commit(&kv_empty[v_slot], leader);
          if (j + 1 < w.last) {
            attn_commit(&kv_empty[ring.slot], leader);
            ring.next();
          }
        }
      }
      if (!ok) {  // the products under way end before their memory is given back
        attn_commit(&drain, leader);
        attn_warp_wait(&drain, 0, status, kDevErrTimeoutFwd);
      }
    }
    __syncwarp();
    }
  } else {
    regs_more<216>();
    // ----------------------------------------------------------------------------- softmax
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t s_col = tc::tmem_lane_addr(tmem, warp, t * 128), o_col = tc::tmem_lane_addr(tmem, warp, Shape::kO + t * DP);
    const float c = d.scale * kLog2e;
    uint32_t parity = 0;  // of s_full; of o_done it is that of the block before
    FwdItem w;
    bool ok = true;
    // (Split: where a wait has run out a warpgroup goes on without waiting, so that the other is not left at their barriers.)
    for (unsigned turn = 0; Split || ok; ++turn) {
      const long long x = attn_item(turn, items, n);
      if (x < 0) break;
      if (!fwd_item<Q>(d, tiles, (unsigned)x, &w)) continue;
      const int first_row = w.i0 + (Split ? 0 : t * kTcBlock), i = first_row + row, off = w.s.m - w.s.n;
      int lo = w.lo[0], hi = w.hi[0];  // Split: the lane's of them, from begin on
      if (!Split && t == 1) lo = w.lo[1], hi = w.hi[1];
      const int begin = Split ? lo + 2 * rank + t : lo;
      // the keys [from, to) that this query sees
      const int from = d.window ? max(0, i + off - d.window + 1) : 0, to = d.causal ? min(w.s.m, i + off + 1) : w.s.m;
      // blocks [clear, full) are seen whole by all of the tile's queries
      const int i_first = first_row, i_last = i_first + kTcBlock - 1;
      const int whole_to = (d.causal ? min(w.s.m, i_first + off + 1) : w.s.m), whole_from = d.window ? i_last + off - d.window + 1 : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = begin; j < hi && ok; j += Split ? 2 * n : 1) {
        ok = attn_warp_wait(&s_full[t], parity, status, kDevErrTimeoutFwd);
        if (!ok) break;
        tc::tc_fence_after();
        float s[128];
#pragma unroll
        for (int e = 0; e < 128; e += 32) tc::tmem_ld32(s_col + e, s + e);
        tc::tmem_wait_ld();
        const int j0 = j * kTcBlock;
        if (j0 + kTcBlock > whole_to || j0 < whole_from) {
          const int a0 = from - j0, a1 = to - j0;
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] = e >= a0 && e < a1 ? s[e] : -INFINITY;
        }
        float tops[4] = {m, m, m, m};  // four chains: one alone is 64 steps long
#pragma unroll
        for (int e = 0; e < 128; e += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) tops[y] = fmaxf(tops[y], fmaxf(s[e + 2 * y], s[e + 2 * y + 1]));
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        if (j == begin) {
          m = top;
        } else {
          const bool grown = (top - m) * c > 8.f;
          if (__any_sync(0xffffffffu, grown)) {
            const float f = grown ? ex2f((m - top) * c) : 1.f;  // of nothing seen before: 0
            if (grown) m = top;
            l *= f;
            ok = attn_warp_wait(&o_done[t], parity ^ 1u, status, kDevErrTimeoutFwd);
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int e = 0; e < DP; e += 16) {
              float o[16];
              uint32_t r[16];
              tc::tmem_ld16(o_col + e, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) r[y] = __float_as_uint(o[y] * f);
              tc::tmem_st16(o_col + e, r);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m * c;
        const f32x2 c2 = pack2(c, c), base2 = pack2(-base, -base);
        f32x2 sum[4] = {0, 0, 0, 0};  // pairs of zeros
#pragma unroll
        for (int e = 0; e < 128; e += 64) {
          uint32_t r[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            const f32x2 p2 = ex2_2(fma2(pack2(s[e + 2 * y], s[e + 2 * y + 1]), c2, base2));
            sum[y & 3] = add2(sum[y & 3], p2);
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo2(p2), hi2(p2));
            r[y] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tc::tmem_st32(s_col + e / 2, r);
          if (e == 0) {  // the product with the first half of the values may begin
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            GDR_DELAY_WARP(56);
            if (lane == 0) tc::mbar_arrive(&p_half[t]);
          }
        }
        const f32x2 both = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += lo2(both) + hi2(both);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        GDR_DELAY(40);
        if (lane == 0) tc::mbar_arrive(&p_ready[t]);
        parity ^= 1u;
      }
      if (!Split && !ok) break;
      const bool mine = i < w.s.n;
      __nv_bfloat16* const out = (__nv_bfloat16*)a.o + ((w.s.q0 + i) * d.Hq + w.h) * (long long)d.D;
      if (begin < hi) {
        ok = ok && attn_warp_wait(&o_done[t], parity ^ 1u, status, kDevErrTimeoutFwd);
        if (!Split && !ok) break;
        tc::tc_fence_after();
      }
      if constexpr (Split) {  // every thread joins its query's two lanes for half of the features
        float(&of)[2][NT][kTcBlock] = joint[turn & 1];
        GDR_DELAY_WARP(60);
        of[0][t][row] = m;
        of[1][t][row] = l;
        tc::tc_fence_before();
        tc::named_sync(1, 2 * kTcBlock);
        tc::tc_fence_after();
        const float m0 = of[0][0][row], m1 = of[0][1][row], top = fmaxf(m0, m1);
        const float f0 = m0 == -INFINITY ? 0.f : ex2f((m0 - top) * c), f1 = m1 == -INFINITY ? 0.f : ex2f((m1 - top) * c);
        const float sum = fmaf(of[1][0][row], f0, of[1][1][row] * f1);
        const int f = t * (DP / 2);
        const uint32_t o0 = tc::tmem_lane_addr(tmem, warp, Shape::kO + f), o1 = tc::tmem_lane_addr(tmem, warp, Shape::kO + DP + f);
        const bool any0 = lo + 2 * rank < hi, any1 = lo + 2 * rank + 1 < hi;
        if constexpr (Share) {
          put_part<DP, DP / 2>(part, row, f, o0, o1, f0, f1, any0, any1);
          if (t == 0) {  // to the second set, which one item leaves unused
            joint[Split][0][0][row] = top;
            joint[Split][1][0][row] = sum;
          }
          continue;
        }
        const bool none = top == -INFINITY && sum == 0.f;  // (scores that are all NaN leave the maximum at -infinity, too)
        const float by = none ? 0.f : 1.f / sum;
        attn_store_row<DP / 2>(o0, o1, out + f, d.D - f, f0 * by, f1 * by, any0, any1, mine);
        if (mine && t == 0) a.lse[w.s.lse0 + (long long)w.h * d.Tq + i] = none ? -INFINITY : fmaf(top, d.scale, logf(sum));
        tc::tc_fence_before();
        tc::named_sync(1, 2 * kTcBlock);  // both lanes' O are read before either is begun anew
      } else {
        // a query that has seen nothing has l = 0 and O = 0 or, where a product has not begun, none (one whose scores are all NaN has
        // the maximum of the first, and l = NaN)
        const bool none = m == -INFINITY && l == 0.f;
        attn_store_row<DP>(o_col, out, d.D, none ? 0.f : 1.f / l, lo < hi, mine);
        if (mine) a.lse[w.s.lse0 + (long long)w.h * d.Tq + i] = none ? -INFINITY : fmaf(m, d.scale, logf(l));
      }
      tc::tc_fence_before();  // O is read before this item's successor's first product into it, which the next arrival allows
    }
  }
  if constexpr (Share) {  // the cluster's one item: every block has its share of the queries
    __syncwarp();
    GDR_DELAY_WARP(61);
    tc::cluster_sync();
    FwdItem w;
    const long long x = attn_item(0, items, n);
    if (warp < 4 * NT && x >= 0 && fwd_item<Q>(d, tiles, (unsigned)x, &w)) {
      const int r0 = kTcBlock * rank / n, r1 = min(kTcBlock * (rank + 1) / n, w.s.n - w.i0);
      const float c = d.scale * kLog2e;
      for (int e = threadIdx.x; e < (r1 - r0) * (DP / 4); e += 2 * kTcBlock) {
        const int r = r0 + e / (DP / 4), piece = e % (DP / 4), i = w.i0 + r;
        float top = -INFINITY, sum = 0.f;
        for (int y = 0; y < n; ++y) top = fmaxf(top, load_peer(&joint[Split][0][0][r], y));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int y = 0; y < n; ++y) {
          const float m = load_peer(&joint[Split][0][0][r], y), f = m == -INFINITY ? 0.f : ex2f((m - top) * c);
          const float4 v = load_peer4(part + part_at<DP>(r, piece), y);
          sum = fmaf(load_peer(&joint[Split][1][0][r], y), f, sum);
          o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        }
        const bool none = top == -INFINITY && sum == 0.f;
        const float by = none ? 0.f : 1.f / sum;
        if (4 * piece < d.D)
          store4((__nv_bfloat16*)a.o + ((w.s.q0 + i) * d.Hq + w.h) * (long long)d.D + 4 * piece,
                 none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * by, o.y * by, o.z * by, o.w * by));
        if (piece == 0) a.lse[w.s.lse0 + (long long)w.h * d.Tq + i] = none ? -INFINITY : fmaf(top, d.scale, logf(sum));
      }
    }
    __syncwarp();
    tc::cluster_sync();  // no block ends while others read it
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 4 * NT) tc::tmem_dealloc(tmem, 512);
}

template <int DP, bool Split>
cudaError_t fwd(const AttnDims& d, const AttnTiles& t, const AttnFwdArgs& a, cudaStream_t s) {
  using Shape = FwdShape<DP, Split>;
  FwdMaps maps;
  const long long rows_q = (long long)d.B * d.Tq, rows_k = (long long)d.B * d.Tk;
  if (!attn_map(&maps.q, a.q, d.D, d.Hq, rows_q, d.ld_q) || !attn_map(&maps.k, a.k, d.D, d.Hk, rows_k, d.ld_k) ||
      !attn_map(&maps.v, a.v, d.D, d.Hk, rows_k, d.ld_v))
    return cudaErrorInvalidValue;
  const long long items = attn_tile_count(d, false, Shape::kQ * kTcBlock) * d.Hq;
  const int n = Split ? attn_sharers(items, (d.Tk + 2 * kTcBlock - 1) / (2 * kTcBlock)) : 1;
  const auto kernel = n > 1 ? attn_fwd_tc_kernel<DP, Split, Split> : attn_fwd_tc_kernel<DP, Split, false>;
  cudaError_t e = set_smem_once((const void*)kernel, Shape::kSmem);
  if (e != cudaSuccess) return e;
  e = attn_launch(kernel, n > 1 ? items * n : std::min<long long>(items, kSmCount), Shape::kThreads, Shape::kSmem, n, s, maps, d, t, (unsigned)items, a);
  if (e != cudaSuccess) return e;
  stage_mark(s, "attn_fwd");
  return cudaGetLastError();
}

}  // namespace

int attn_fwd_tc_tile(const AttnDims& d) {
  return attn_tile_count(d, false, 2 * kTcBlock) * d.Hq >= kSmCount ? 2 * kTcBlock : kTcBlock;
}

cudaError_t launch_attn_fwd_tc(const AttnDims& d, const AttnTiles& t, int tile, const AttnFwdArgs& a, cudaStream_t s) {
  if (tile == 2 * kTcBlock) return d.D > 64 ? fwd<128, false>(d, t, a, s) : fwd<64, false>(d, t, a, s);
  return d.D > 64 ? fwd<128, true>(d, t, a, s) : fwd<64, true>(d, t, a, s);
}

}  // namespace gdr
