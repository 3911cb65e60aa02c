// gdr_attn_step.cu -- attention of one token per sequence over a paged cache, and the write of a prompt into it
// (include/gdr_attn.h).
//
// The step reads the visible part of the cache once and is bound by that.  The work is the list of all tiles of 64
// (bf16) or 32 (fp32) positions of all rows and key heads, one behind the other, each (row, key head) with one more place for what
// beginning and ending it costs; a launch of two blocks per SM cuts the list into equal parts, so that one long sequence, many short
// ones and any mixture of them load every SM alike.  Which rows have how many tiles is on the device only (lengths): every block sums
// them up itself.  A block takes its tiles in order.  One warp
// has TMA bring them into a ring of three stages (128 KB per SM under way): boxes of as many positions of a page as a power of two
// divides its size by, at most a tile.  Four warps keep the running maximum m, sum l and O of a (row, key head), for up to 16
// query heads that share it:
//   bf16: mma.m16n8k16, query heads as the rows, so that P's accumulator is the next product's operand; a warp takes 16 of a
//         tile's positions.  The products are small beside the copies (16 rows of 16 positions of 128 features: 32 instructions).
//   fp32: on the FMA pipes, 4 lanes per position for S, 4 features per lane for O.
// A (row, key head) that lies within one block is finished there; of the others each block leaves its part (m, l, O), and a
// second launch adds them in order.  Short rows change every tile: whatever a unit needs (its queries, its new token) comes
// through the ring with its tiles, and its warps' parts are added in the stage that its last tile had.  The new token's key and value
// go from the call's inputs to shared memory and the cache; what a page holds outside a row's visible positions is replaced by zeros there.
// bf16, pages of 64: 64 rows of up to 8192 positions, 32 heads on 8 of 128: 117 to 121 us, 6.0 TB/s (437 us and more before what a unit needs
// came through the ring); 40 heads on 8: 123.  fp32, 32 heads on 8: 247 us, 5.8 TB/s, but 40 on 8: 1242 us, 1.2 TB/s (above four query heads a
// unit's arithmetic is that of sixteen, one block per SM, and binds).  One row of 65536: 31 us, of which about 8 are set-up and the join (with
// eight parts' loads a warp, begun behind the maxima, 6 us more).  With 16-byte copies by all threads the latter took 84 us (1000 instructions a
// tile and warp), with a bulk copy for every position 96 (41 cycles a copy, one after the other).
#include <cmath>
#include <cstring>

#include "gdr_attn.cuh"
#include "gdr_instrument.cuh"
#include "tc_primitives.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;  // that compute; a warp more copies
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 3;
constexpr int kHeads = 16;  // query heads of a unit

struct StepDims {
  int B, Hq, Hk, D, G, HB;  // HB: units per key head
  int num_pages, page_size, max_pages;
  int window;
  float scale;
  long long ld_q, ld_k, ld_v;
  int vec;  // q, k, v by 16 bytes
  int box;  // positions of a copy
};

struct StepMaps {
  CUtensorMap k, v;
};

// A stage: K then V, each in slabs of 128 bytes of every position's features, 16-byte chunks swizzled by the position.
template <typename IT> constexpr int slab_features() { return 128 / (int)sizeof(IT); }

// Positions that a tile covers.
template <typename IT> constexpr int tile_keys() { return sizeof(IT) == 2 ? 64 : 32; }
template <typename IT> constexpr int slab_bytes() { return tile_keys<IT>() * 128; }
// Byte offset of 16-byte chunk `c` of position `r` in a K or V tile.
template <typename IT>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * slab_bytes<IT>() + r * 128 + (((c ^ r) & 7) << 4));
}

// The visible positions lo .. len of a row and its tiles; false: the row is skipped.
struct Row {
  int len, lo, tile0, tiles;
  __device__ __forceinline__ int places() const { return tiles ? tiles + 1 : 0; }  // in the list, of each unit
};
template <int KT>
__device__ __forceinline__ Row row_of(const StepDims& d, const int32_t* lengths, int b) {
  Row r;
  r.len = lengths[b];
  const bool ok = r.len >= 0 && r.len < (long long)d.max_pages * d.page_size;
  r.lo = d.window ? max(0, r.len - d.window + 1) : 0;
  r.tile0 = r.lo / KT;
  r.tiles = ok ? r.len / KT - r.tile0 + 1 : 0;
  return r;
}

// Places of one unit of the rows before thread t's rows (B cut into kThreads runs), and of all: prefix[kThreads + 1] in shared memory.
template <int KT>
__device__ __forceinline__ void sum_rows(const StepDims& d, const int32_t* lengths, long long* prefix) {
  const int tid = threadIdx.x, run = (d.B + kThreads - 1) / kThreads;
  const bool on = tid < kThreads;
  long long sum = 0;
  if (on)
    for (int b = tid * run; b < min(d.B, (tid + 1) * run); ++b) sum += row_of<KT>(d, lengths, b).places();
  long long v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if ((tid & 31) >= o) v += y;
  }
  if (on) prefix[tid + 1] = v;  // within the warp
  if (tid == 0) prefix[0] = 0;
  __syncthreads();
  long long before = 0;
  for (int w = 0; w < (tid >> 5) && on; ++w) before += prefix[32 * (w + 1)];
  __syncthreads();
  if (on) prefix[tid + 1] = v + before;
  __syncthreads();
}

// A place in the list: row, unit of the row (key head and block of query heads), tile of the unit (-1: the place in front of it).
template <int KT>
struct Cursor {
  int b, unit, tile;
  Row row;
  __device__ __forceinline__ void seek(const StepDims& d, const int32_t* lengths, const long long* prefix, int units, long long at) {
    int lo = 0, hi = kThreads - 1;  // the last run that begins at or before the place
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] * units <= at) lo = mid; else hi = mid - 1;
    }
    long long rest = at - prefix[lo] * units;
    b = lo * ((d.B + kThreads - 1) / kThreads);
    row = row_of<KT>(d, lengths, b);
    while (rest >= (long long)row.places() * units) {
      rest -= (long long)row.places() * units;
      row = row_of<KT>(d, lengths, ++b);
    }
    unit = (int)(rest / row.places());
    tile = (int)(rest % row.places()) - 1;
  }
  // The next tile, if there is one before place `end`; `at` is the place it is at.
  __device__ __forceinline__ bool next(const StepDims& d, const int32_t* lengths, int units, long long* at, long long end) {
    const bool within = tile + 1 < row.tiles;
    *at += within ? 1 : 2;
    if (*at >= end) return false;
    if (within) {
      ++tile;
      return true;
    }
    tile = 0;
    if (++unit == units) {
      unit = 0;
      do row = row_of<KT>(d, lengths, ++b);
      while (row.tiles == 0);
    }
    return true;
  }
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A box of a cache: features f .., one head, positions place .. of a page.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint64_t* bar, int f, int h, int place, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(f), "r"(h), "r"(place), "r"(page), "r"(smem_addr(bar))
      : "memory");
}

// The larger, or a NaN where there is one: it has to reach the row's result.
__device__ __forceinline__ float max_nan(float a, float b) { return b > a || b != b ? b : a; }

// A bounded wait by a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, status, kDevErrTimeoutFwd));
}

// Running softmax of a warp's part of the tiles, products on the tensor cores.
template <int DP>
struct EngineBf16 {
  static constexpr int kBlocks = 2;     // per SM
  uint32_t qa[DP / 16][4];
  float O[DP / 8][4], m[2], l[2];  // heads lane / 4 and lane / 4 + 8; m in units of S

  __device__ __forceinline__ void begin(const __nv_bfloat16* q, int heads, int D) {  // q: shared memory [heads][D]
    const int lane = threadIdx.x & 31, g = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = g + 8 * (i & 1), f = 16 * kk + c + 8 * (i >> 1);
        qa[kk][i] = r < heads && f < D ? *reinterpret_cast<const uint32_t*>(q + r * D + f) : 0u;
      }
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[n][i] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // The warp's 16 positions of a tile whose first position is p0.
  __device__ __forceinline__ void tile(const unsigned char* K, const unsigned char* V, int p0, const Row& row, float c) {
    using IT = __nv_bfloat16;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t ka = smem_addr(K);
    const int kr = 16 * w + (lane & 7) + 8 * (lane >> 4);
    float s[2][4] = {}, s2[2][4] = {};  // even and odd steps: two chains of products at a time are too few
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      uint32_t b[4];
      ldmatrix4(b, ka + chunk_at<IT>(kr, 2 * kk + (lane >> 3 & 1)));
      mma16816(kk & 1 ? s2[0] : s[0], qa[kk], b[0], b[1]);
      mma16816(kk & 1 ? s2[1] : s[1], qa[kk], b[2], b[3]);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] += s2[n][i];
    const int at = p0 + 16 * w + 2 * (lane & 3);
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = at + 8 * n + (i & 1);
        if (p < row.lo || p > row.len) s[n][i] = -INFINITY;
        top[i >> 1] = max_nan(top[i >> 1], s[n][i]);
      }
    uint32_t pa[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = max_nan(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = max_nan(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float base = attn_base(top[r], c), f = attn_rescale(m[r], c, base);
      m[r] = top[r];
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0_ = ex2f(fmaf(s[n][2 * r], c, -base)), p1_ = ex2f(fmaf(s[n][2 * r + 1], c, -base));
        sum += p0_ + p1_;
        pa[2 * n + r] = pack_bf16(p0_, p1_);
      }
      l[r] = fmaf(l[r], f, sum);
      if (__any_sync(0xffffffffu, f != 1.f))
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          O[n][2 * r] *= f;
          O[n][2 * r + 1] *= f;
        }
    }
    const uint32_t va = smem_addr(V);
    const int vr = 16 * w + (lane & 15);
#pragma unroll
    for (int n = 0; n < DP / 16; ++n) {
      uint32_t b[4];
      ldmatrix4t(b, va + chunk_at<IT>(vr, 2 * n + (lane >> 4)));
      mma16816(O[2 * n], pa, b[0], b[1]);
      mma16816(O[2 * n + 1], pa, b[2], b[3]);
    }
  }

  __device__ __forceinline__ void stats(float* ms, float* ls, int) {  // [kHeads] of this warp
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        ms[(lane >> 2) + 8 * r] = m[r];
        ls[(lane >> 2) + 8 * r] = l[r];
      }
    }
  }
  // acc[head][feature] = O f(head) of the heads.
  template <typename F>
  __device__ __forceinline__ void put(float* acc, int heads, F f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int head = (lane >> 2) + 8 * r;
      if (head >= heads) continue;
      const float by = f(head);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
        *reinterpret_cast<float2*>(acc + head * DP + 8 * n + 2 * (lane & 3)) = make_float2(O[n][2 * r] * by, O[n][2 * r + 1] * by);
    }
  }
};

// The same in fp32; NH: query heads that it is built for (at least the unit's).
template <int DP, int NH>
struct EngineF32 {
  static constexpr int kBlocks = NH == kHeads ? 1 : 2;
  static constexpr int F = DP / 32;  // features of O per lane: F lane ..
  const float* q;                    // shared memory [heads][D]
  int heads, D;
  float O[NH][F], m[NH], l[NH];

  __device__ __forceinline__ void begin(const float* from, int heads_, int D_) {
    q = from;
    heads = heads_;
    D = D_;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
#pragma unroll
      for (int i = 0; i < F; ++i) O[r][i] = 0.f;
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
  }
  // The warp's 8 positions of a tile.
  __device__ __forceinline__ void tile(const unsigned char* K, const unsigned char* V, int p0, const Row& row, float c) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, kr = 8 * w + (lane >> 2);
    float s[NH];
#pragma unroll
    for (int r = 0; r < NH; ++r) s[r] = 0.f;
#pragma unroll
    for (int k = 0; k < DP; k += 16) {
      if (k >= D) break;
      const float4 a = *reinterpret_cast<const float4*>(K + chunk_at<float>(kr, k / 4 + (lane & 3)));
#pragma unroll
      for (int r = 0; r < NH; ++r) {
        // (heads behind the unit's last are the last one's copies, whose results are not used)
        const float4 b = *reinterpret_cast<const float4*>(q + min(r, heads - 1) * D + k + 4 * (lane & 3));
        s[r] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s[r]))));
      }
    }
    const int p = p0 + 8 * w + (lane >> 2);
    const bool on = p >= row.lo && p <= row.len;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
      s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
      s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
      if (!on) s[r] = -INFINITY;
      float top = max_nan(m[r], s[r]);
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = attn_base(top, c), f = attn_rescale(m[r], c, base);
      m[r] = top;
      s[r] = ex2f(fmaf(s[r], c, -base));
      l[r] = fmaf(l[r], f, s[r]);  // of the lane's positions
#pragma unroll
      for (int i = 0; i < F; ++i) O[r][i] *= f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[F];
#pragma unroll
      for (int i = 0; i < F; ++i)
        v[i] = reinterpret_cast<const float*>(V + chunk_at<float>(8 * w + j, F * lane / 4))[F * lane % 4 + i];
#pragma unroll
      for (int r = 0; r < NH; ++r) {
        const float pj = __shfl_sync(0xffffffffu, s[r], 4 * j);
#pragma unroll
        for (int i = 0; i < F; ++i) O[r][i] = fmaf(pj, v[i], O[r][i]);
      }
    }
  }
  __device__ __forceinline__ void stats(float* ms, float* ls, int) {
#pragma unroll
    for (int r = 0; r < NH; ++r) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
      if ((threadIdx.x & 31) == 0) {
        ms[r] = m[r];
        ls[r] = l[r];
      }
    }
  }
  template <typename Fn>
  __device__ __forceinline__ void put(float* acc, int, Fn f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
      if (r >= heads) break;
      const float by = f(r);
#pragma unroll
      for (int i = 0; i < F; ++i) acc[r * DP + F * lane + i] = O[r][i] * by;
    }
  }
};

template <typename IT, int DP>
constexpr size_t stage_bytes() { return 2 * sizeof(IT) * tile_keys<IT>() * DP; }
// Beside a stage: the queries of the unit that begins with its tile, and the new token of the one that ends with it.
template <typename IT, int DP>
constexpr size_t side_bytes(int rows) { return sizeof(IT) * DP * (rows + 2); }
template <typename IT, int DP>  // room to align, then the stages and what is beside them; fp32: the queries of the unit in work
constexpr size_t step_smem(int rows) {
  return 1024 + kStages * (stage_bytes<IT, DP>() + side_bytes<IT, DP>(rows)) + (sizeof(IT) == 4 ? sizeof(IT) * DP * rows : 0);
}
// A part: O [kHeads][DP], m [kHeads], l [kHeads] (l < 0: the row needs a page outside the pool).
template <int DP>
constexpr int part_floats() { return kHeads * (DP + 2); }

template <typename IT, int DP, typename Engine>
__global__ void __launch_bounds__(kThreads + 32, Engine::kBlocks)
    attn_step_kernel(const __grid_constant__ StepMaps maps, StepDims d, const IT* q, const IT* k,
                     const IT* v, IT* k_cache, IT* v_cache, const int32_t* table,
                     const int32_t* lengths, IT* o, int2* spans, float* parts,
                     uint32_t* status) {
  constexpr int KT = tile_keys<IT>(), N = 16 / (int)sizeof(IT), kSlabs = DP / slab_features<IT>();
  constexpr uint32_t kTileBytes = stage_bytes<IT, DP>() / 2;
  extern __shared__ unsigned char raw[];
  __shared__ long long prefix[kThreads + 1];
  __shared__ float ms[2][kWarps][kHeads], ls[2][kWarps][kHeads];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ int stage_bad[kStages], stage_page[kStages];  // the page that the new token goes to, or -1
  unsigned char* const stages = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, units = d.Hk * d.HB, rows = min(d.G, kHeads);
  // new key, new value, queries
  auto side = [&](int stage) { return reinterpret_cast<IT*>(stages + kStages * stage_bytes<IT, DP>() + stage * side_bytes<IT, DP>(rows)); };
  launch_wait();
  launch_next();
  if (blockIdx.x == 0 && tid == 0) *status = 0;  // (a wait that runs out sets it two seconds later)
  if (tid == kThreads) {
    tc::tma_prefetch_desc(&maps.k);
    tc::tma_prefetch_desc(&maps.v);
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], kWarps);
    }
    tc::fence_barrier_init();
  }
  sum_rows<KT>(d, lengths, prefix);  // its barriers order what is above, too
  const long long total = prefix[kThreads] * units;
  // no more blocks than places: of the blocks between those that have a unit's first and last tile, each has some of its tiles
  const long long blocks = min((long long)gridDim.x, total);
  if (blockIdx.x >= blocks) return;
  const long long start = total * blockIdx.x / blocks, end = total * (blockIdx.x + 1) / blocks;
  Cursor<KT> here;
  here.seek(d, lengths, prefix, units, start);
  long long at = start;
  if (here.tile < 0 && !here.next(d, lengths, units, &at, end)) return;
  long long count = 0;  // tiles so far
  int stage = 0;
  uint32_t parity = 0;

  if (warp == kWarps) {
    // -------------------------------------------------------------------------------- copies
    constexpr int R = KT / 32;  // boxes of a lane at most
    const int boxes = KT / d.box;
    const uint32_t bytes = (uint32_t)d.box * 128;
    // the pages of the lane's boxes of a tile: -1 for positions that are not seen or only written, -2 for a page outside the pool
    auto pages_of = [&](int (&pages)[R]) {
      const int p0 = (here.row.tile0 + here.tile) * KT, first = p0 / d.page_size, rest = p0 - first * d.page_size;
      const int32_t* at = table + (long long)here.b * d.max_pages + first;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int x = lane + 32 * i, r = x * d.box, y = rest + r;
        pages[i] = -1;
        if (x >= boxes || p0 + r + d.box <= here.row.lo || p0 + r > here.row.len) continue;
        const int page = at[d.page_size >= KT ? (int)(y >= d.page_size) : y / d.page_size];
        pages[i] = page < 0 || page >= d.num_pages ? -2 : p0 + r == here.row.len ? -1 : page;
      }
    };
    auto new_page = [&]() {  // of a unit's last tile, one unit of a key head
      if (here.tile + 1 < here.row.tiles || here.unit % d.HB != 0) return -1;
      const int page = table[(long long)here.b * d.max_pages + here.row.len / d.page_size];
      return page >= 0 && page < d.num_pages ? page : -1;
    };
    int pages[R];
    pages_of(pages);
    int into = new_page();
    for (bool more = true; more; ++count) {
      const int h = here.unit / d.HB, hb = here.unit % d.HB, b = here.b, rest = (here.row.tile0 + here.tile) * KT % d.page_size;
      const bool begins = count == 0 || here.tile == 0, ends = here.tile + 1 == here.row.tiles;
      int from[R], place[R];
      bool bad = false;
      int copies = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int y = rest + (lane + 32 * i) * d.box;
        place[i] = d.page_size >= KT ? (y >= d.page_size ? y - d.page_size : y) : y % d.page_size;
        from[i] = pages[i];
        bad |= pages[i] == -2;
        copies += __popc(__ballot_sync(0xffffffffu, pages[i] >= 0));
      }
      bad = __any_sync(0xffffffffu, bad);
      const int page = into;
      more = here.next(d, lengths, units, &at, end);
      if (more) {  // the next tile's pages are on their way while this one's copies are issued
        pages_of(pages);
        into = new_page();
      }
      if (!attn_wait(&empty[stage], parity ^ 1u, status)) break;
      GDR_DELAY_WARP(50);
      unsigned char* const ks = stages + (size_t)stage * stage_bytes<IT, DP>();
      IT* const beside = side(stage);
      const int heads = min(kHeads, d.G - hb * kHeads);
      const IT* const qf = q + (long long)b * d.ld_q + (long long)(h * d.G + hb * kHeads) * d.D;
      const IT *const kf = k + (long long)b * d.ld_k + (long long)h * d.D, *const vf = v + (long long)b * d.ld_v + (long long)h * d.D;
      const uint32_t row_bytes = (uint32_t)d.D * sizeof(IT);
      uint32_t extra = 0;
      if (d.vec) {
        extra = (begins ? heads * row_bytes : 0u) + (ends ? 2 * row_bytes : 0u);
      } else {  // not aligned for bulk copies
        if (begins)
          for (int i = lane; i < heads * d.D; i += 32) beside[2 * DP + i] = qf[i];
        if (ends)
          for (int i = lane; i < d.D; i += 32) beside[i] = kf[i], beside[DP + i] = vf[i];
        __syncwarp();
      }
      if (lane == 0) {
        stage_bad[stage] = bad;
        stage_page[stage] = page;
        tc::mbar_arrive_expect_tx(&full[stage], 2 * kSlabs * bytes * copies + extra);
        if (d.vec && begins) tc::bulk_load(beside + 2 * DP, qf, heads * row_bytes, &full[stage]);
        if (d.vec && ends) {
          tc::bulk_load(beside, kf, row_bytes, &full[stage]);
          tc::bulk_load(beside + DP, vf, row_bytes, &full[stage]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (from[i] >= 0) {
          unsigned char* const to = ks + (lane + 32 * i) * bytes;
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl) {
            load_box(to + sl * slab_bytes<IT>(), &maps.k, &full[stage], sl * slab_features<IT>(), h, place[i], from[i]);
            load_box(to + kTileBytes + sl * slab_bytes<IT>(), &maps.v, &full[stage], sl * slab_features<IT>(), h, place[i], from[i]);
          }
        }
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }
    // every copy is waited for by the warps that compute; should one of their waits have run out, here
    for (int i = 0; i < kStages; ++i) {
      if (count > i) attn_wait(&full[i], (uint32_t)((count - 1 - i) / kStages) & 1u, status);
    }
    return;
  }

  Engine e;
  const float c = d.scale * kLog2e;
  int first_tile = here.tile, heads = 0, ended = 0;  // ended: units, or parts of one, so far
  // Where a wait has run out the block goes on without waiting, so that no warp is left at a barrier; its results are lost.
  bool fresh = true, bad = false, ok = true;
  for (bool more = true; more;) {
    ok = ok && attn_wait(&full[stage], parity, status);
    GDR_DELAY_WARP(51);
    unsigned char* const ks = stages + (size_t)stage * stage_bytes<IT, DP>();
    unsigned char* const vs = ks + kTileBytes;
    const IT* const beside = side(stage);
    if (fresh) {
      heads = min(kHeads, d.G - here.unit % d.HB * kHeads);
      if constexpr (sizeof(IT) == 4) {  // read all through the unit, while the stage goes on to others
        IT* const qs = side(kStages);
        for (int i = tid; i < heads * d.D; i += kThreads) qs[i] = beside[2 * DP + i];
        tc::named_sync(1, kThreads);
        e.begin(qs, heads, d.D);
      } else {
        e.begin(beside + 2 * DP, heads, d.D);
      }
      first_tile = here.tile;
      fresh = bad = false;
    }
    const int p0 = (here.row.tile0 + here.tile) * KT;
    const bool edge = p0 < here.row.lo || p0 + KT > here.row.len;
    if (edge) {  // of the warp's own positions: values that are not seen become zeros, the new token comes to its place
      constexpr int W = KT / kWarps, C = DP / N;
      for (int x = lane; x < W * C; x += 32) {
        const int r = W * warp + x / C, p = p0 + r;
        if (p < here.row.lo || p > here.row.len) *reinterpret_cast<uint4*>(vs + chunk_at<IT>(r, x % C)) = make_uint4(0, 0, 0, 0);
      }
      const int r = here.row.len - p0;
      if (r / W == warp && r < KT && lane < C) {
        const bool on = lane * N < d.D;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 kn = on ? reinterpret_cast<const uint4*>(beside)[lane] : zero, vn = on ? reinterpret_cast<const uint4*>(beside + DP)[lane] : zero;
        *reinterpret_cast<uint4*>(ks + chunk_at<IT>(r, lane)) = kn;
        *reinterpret_cast<uint4*>(vs + chunk_at<IT>(r, lane)) = vn;
        if (stage_page[stage] >= 0 && on) {
          const long long to = (((long long)stage_page[stage] * d.page_size + here.row.len % d.page_size) * d.Hk + here.unit / d.HB) * d.D + lane * N;
          *reinterpret_cast<uint4*>(k_cache + to) = kn;
          *reinterpret_cast<uint4*>(v_cache + to) = vn;
        }
      }
      __syncwarp();
    }
    e.tile(ks, vs, p0, here.row, c);
    bad |= stage_bad[stage] != 0;
    Cursor<KT> then = here;
    more = then.next(d, lengths, units, &at, end);
    const bool last = here.tile + 1 == here.row.tiles || !more;  // of a (row, unit), or of the block's part of it
    if (last) {
      GDR_DELAY_WARP(52);
      float(&m_of)[kWarps][kHeads] = ms[ended & 1], (&l_of)[kWarps][kHeads] = ls[ended & 1];  // (a warp that is one unit on writes to the others)
      e.stats(m_of[warp], l_of[warp], heads);
      tc::named_sync(1, kThreads);  // from here on no warp reads the tile: its stage takes the warps' parts
      float* const acc = reinterpret_cast<float*>(ks);
      auto top_of = [&](int r) { return max_nan(max_nan(m_of[0][r], m_of[1][r]), max_nan(m_of[2][r], m_of[3][r])); };
      auto share = [&](int w, int r) { return attn_rescale(m_of[w][r], c, attn_base(top_of(r), c)); };  // of warp w's part in the whole
      e.put(acc + warp * kHeads * DP, heads, [&](int r) { return share(warp, r); });
      GDR_DELAY_WARP(53);
      tc::named_sync(1, kThreads);
      GDR_DELAY_WARP(54);
      const bool whole = first_tile == 0 && here.tile + 1 == here.row.tiles;
      const int slot = ended++ > 0 ? 1 : 0;
      float* const part = parts + ((long long)blockIdx.x * 2 + slot) * part_floats<DP>();
      if (tid == 0) {  // which blocks have the unit's parts
        int2* const span = spans + (long long)here.b * units + here.unit;
        if (first_tile == 0) span->x = whole ? -1 : (int)blockIdx.x * 2 + slot;
        if (here.tile + 1 == here.row.tiles) span->y = (int)blockIdx.x;
      }
      for (int r = warp; r < heads; r += kWarps) {  // a warp per head, DP / 32 features per lane
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l = fmaf(l_of[w][r], share(w, r), l);
        const float by = 1.f / l;
        const int h = here.unit / d.HB * d.G + here.unit % d.HB * kHeads + r;
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          const int f = 32 * i + lane;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum += acc[(w * kHeads + r) * DP + f];
          if (!whole)
            part[r * DP + f] = sum;
          else if (f < d.D)
            o[((long long)here.b * d.Hq + h) * d.D + f] = from_f32<IT>(bad ? 0.f : sum * by);
        }
        if (!whole && lane == 0) {
          part[kHeads * DP + r] = top_of(r);
          part[kHeads * (DP + 1) + r] = bad ? -1.f : l;
        }
      }
      fresh = true;
    }
    if (edge || last) tc::fence_proxy_async_smem();  // a later round's copies come to the same places
    __syncwarp();
    GDR_DELAY_WARP(55);
    if (lane == 0) tc::mbar_arrive(&empty[stage]);
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1u;
    }
    here = then;
  }
}

// The rows' results that several blocks have parts of, and zeros for the rows that were skipped.  A block per query head of a row;
// a warp has Ahead parts' loads under way, the first ones' while the largest maximum is looked for.  Bound by latency.
template <typename IT, int DP, int Ahead>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(StepDims d, const int32_t* lengths, IT* o,
                                                             const int2* spans, const float* parts) {
  __shared__ float red[kWarps][2];
  __shared__ float total_of[kWarps][DP];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = (int)(blockIdx.x / (unsigned)d.Hq), h = (int)(blockIdx.x % (unsigned)d.Hq);
  const int r = h % d.G % kHeads;
  launch_wait();
  launch_next();
  const int2 span = spans[((long long)b * d.Hk + h / d.G) * d.HB + h % d.G / kHeads];  // (not written for a row that was skipped)
  const Row row = row_of<tile_keys<IT>()>(d, lengths, b);
  IT* out = o + ((long long)b * d.Hq + h) * d.D;
  if (row.tiles == 0) {
    if (tid < d.D) out[tid] = from_f32<IT>(0.f);
    return;
  }
  if (span.x < 0) return;
  // the first block's part is its second where another unit's came before it; the later blocks begin within this unit
  const int c0 = span.x >> 1, c1 = span.y;
  auto part_of = [&](int x) { return parts + ((long long)x * 2 + (x == c0 ? span.x & 1 : 0)) * part_floats<DP>(); };
  const float c = d.scale * kLog2e;
  // a warp takes every fourth part, a lane DP / 32 features
  constexpr int F = DP / 32;
  float v[Ahead][F], pm[Ahead], pl[Ahead];
  auto load = [&](int x0) {
#pragma unroll
    for (int i = 0; i < Ahead; ++i) {
      const int x = x0 + i * kWarps;
      if (x > c1) break;
      const float* p = part_of(x);
      pm[i] = p[kHeads * DP + r];
      pl[i] = p[kHeads * (DP + 1) + r];
#pragma unroll
      for (int f = 0; f < F; ++f) v[i][f] = p[r * DP + F * lane + f];
    }
  };
  load(c0 + warp);
  // the largest maximum, and whether a part is bad
  float top = -INFINITY, bad = 0.f;
  for (int x = c0 + tid; x <= c1; x += kThreads) {
    const float* p = part_of(x);
    top = max_nan(top, p[kHeads * DP + r]);
    bad = p[kHeads * (DP + 1) + r] < 0.f ? 1.f : bad;
  }
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, x));
    bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, x));
  }
  if ((tid & 31) == 0) {
    red[tid >> 5][0] = top;
    red[tid >> 5][1] = bad;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    top = max_nan(top, red[w][0]);
    bad = fmaxf(bad, red[w][1]);
  }
  __syncthreads();  // red is used again
  const float base = attn_base(top, c);
  float sum[F] = {}, l = 0.f;
  for (int x0 = c0 + warp; x0 <= c1; x0 += Ahead * kWarps) {
    if (x0 > c0 + warp) load(x0);
#pragma unroll
    for (int i = 0; i < Ahead; ++i) {
      if (x0 + i * kWarps > c1) break;
      const float weight = attn_rescale(pm[i], c, base);
      l = fmaf(pl[i], weight, l);
#pragma unroll
      for (int f = 0; f < F; ++f) sum[f] = fmaf(v[i][f], weight, sum[f]);
    }
  }
  // then the warps' sums in order
#pragma unroll
  for (int f = 0; f < F; ++f) total_of[warp][F * lane + f] = sum[f];
  if (lane == 0) red[warp][0] = l;
  __syncthreads();
  if (tid < d.D) {
    float a0 = 0.f, l0 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a0 += total_of[w][tid];
      l0 += red[w][0];
    }
    out[tid] = from_f32<IT>(bad > 0.f ? 0.f : a0 / l0);
  }
}

// ------------------------------------------------------------------------------ prompts to pages
// A copy, bound by memory.  A thread takes kPieces times 16 bytes of one token, of k and of v: what it looks up (sequence, place,
// page) serves all of them, and their loads are under way together.  Eight prompts, 234 MB read and written: 37 us, 6.3 TB/s (3 us more with one piece);
// element by element, where k or v is off 16 bytes, 93 us.
constexpr int kPieces = 2;
struct WriteDims {
  int B, T, Hk, D, num_pages, page_size, max_pages;
  const int32_t* cu;
  long long tokens, ld_k, ld_v;
};

template <typename IT, int V>
__global__ void __launch_bounds__(256) cache_write_kernel(WriteDims d, const IT* k, const IT* v,
                                                          IT* k_cache, IT* v_cache,
                                                          const int32_t* table, const int32_t* starts,
                                                          uint32_t* status) {
  launch_wait();
  launch_next();
  if (d.cu) {
    bool bad = false;
    for (int n = threadIdx.x; n < d.B; n += 256) bad |= d.cu[n] > d.cu[n + 1];
    if (threadIdx.x == 0) bad |= d.cu[0] != 0 || d.cu[d.B] != d.T;
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = bad ? kDevErrBadCuSeqlens : 0u;
    if (bad) return;
  }
  const int wide = d.Hk * d.D / V, part = (wide + kPieces - 1) / kPieces;  // pieces of a token, of them a thread's distance
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x, token = x / part;
  if (token >= d.tokens) return;
  const int c = (int)(x - token * part);
  using Piece = std::conditional_t<V == 1, IT, uint4>;
  Piece a[kPieces], b[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = c + i * part;
    if (e >= wide) break;
    const Piece *ka = reinterpret_cast<const Piece*>(k + token * d.ld_k) + e, *va = reinterpret_cast<const Piece*>(v + token * d.ld_v) + e;
    if constexpr (V == 1) {
      a[i] = *ka;
      b[i] = *va;
    } else {
      a[i] = load_once(ka);
      b[i] = load_once(va);
    }
  }
  const int n = d.cu ? seq_of(d.cu, d.B, token) : (int)(token / d.T);
  const long long t = d.cu ? token - d.cu[n] : token - (long long)n * d.T;
  const long long pos = t + (starts ? starts[n] : 0);
  if (pos < 0 || pos >= (long long)d.max_pages * d.page_size) return;
  const int pi = (int)pos / d.page_size, page = table[(long long)n * d.max_pages + pi];
  if (page < 0 || page >= d.num_pages) return;
  const long long to = ((long long)page * d.page_size + ((int)pos - pi * d.page_size)) * d.Hk * d.D;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = c + i * part;
    if (e >= wide) break;
    reinterpret_cast<Piece*>(k_cache + to)[e] = a[i];
    reinterpret_cast<Piece*>(v_cache + to)[e] = b[i];
  }
}

gdr_status check_cache(const gdr_cache_problem* p, bool step) {
  if (p == nullptr || p->B < 0 || p->T < 0 || p->Hk <= 0 || p->D <= 0 || p->num_pages < 0 || p->page_size <= 0 || p->max_pages < 0)
    return GDR_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || p->ld_q < 0 || p->ld_k < 0 || p->ld_v < 0) return GDR_ERR_INVALID_ARG;
  const long long wk = (long long)p->Hk * p->D;
  if ((p->ld_k && p->ld_k < wk) || (p->ld_v && p->ld_v < wk)) return GDR_ERR_INVALID_ARG;
  if (step) {
    if (p->T != 1 || p->cu_seqlens || p->Hq <= 0 || p->Hq % p->Hk != 0 || p->window < 0 || !std::isfinite(p->scale)) return GDR_ERR_INVALID_ARG;
    if (p->ld_q && p->ld_q < (long long)p->Hq * p->D) return GDR_ERR_INVALID_ARG;
  }
  if (p->D % 16 != 0 || p->D > 128) return GDR_ERR_UNSUPPORTED;
  const long long most = 1ll << 31;
  // positions of a row are 32-bit numbers, as lengths are
  if ((long long)p->max_pages * p->page_size >= most - 256 || wk >= most) return GDR_ERR_UNSUPPORTED;  // (a tile's end fits, too)
  if (step && (long long)p->B * p->Hq >= most) return GDR_ERR_UNSUPPORTED;
  if (wk * p->page_size * (long long)dtype_bytes(p->dtype) >= 1ll << 40) return GDR_ERR_UNSUPPORTED;  // a page, as a stride of TMA
  if (!step && (p->cu_seqlens ? (long long)p->T : (long long)p->B * p->T) >= most) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

struct StepShape {
  StepDims d;
  int blocks;
  size_t spans, bytes;  // bytes: the status word, the spans, the parts
};
StepShape step_shape(const gdr_cache_problem* p) {
  StepShape s;
  const long long wq = (long long)p->Hq * p->D, wk = (long long)p->Hk * p->D;
  const int G = p->Hq / p->Hk, KT = p->dtype == GDR_DTYPE_BF16 ? tile_keys<__nv_bfloat16>() : tile_keys<float>();
  s.d = StepDims{p->B, p->Hq, p->Hk, p->D, G, (G + kHeads - 1) / kHeads, p->num_pages, p->page_size, p->max_pages, p->window,
                 p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)p->D)), p->ld_q ? p->ld_q : wq, p->ld_k ? p->ld_k : wk,
                 p->ld_v ? p->ld_v : wk, 0, 1};
  while (s.d.box < KT && p->page_size % (2 * s.d.box) == 0) s.d.box *= 2;
  const long long most = ((long long)p->max_pages * p->page_size + KT - 1) / KT;  // tiles of a row at most
  const double tiles = (double)p->B * p->Hk * s.d.HB * (double)most;
  s.blocks = tiles < 2 * kSmCount ? (int)tiles : 2 * kSmCount;
  if (s.blocks < 1) s.blocks = 1;
  s.spans = block_align(sizeof(int2) * (size_t)p->B * p->Hk * s.d.HB);
  s.bytes = 256 + s.spans + block_align(sizeof(float) * 2 * (size_t)s.blocks * (p->D > 64 ? part_floats<128>() : part_floats<64>()));
  return s;
}

template <typename IT, int DP, typename Engine>
cudaError_t step(const StepShape& sh, const void* q, const void* k, const void* v, void* kc, void* vc, const int32_t* table,
                 const int32_t* lengths, void* o, void* workspace, cudaStream_t s) {
  uint32_t* const status = (uint32_t*)workspace;
  int2* const spans = (int2*)((char*)workspace + 256);
  float* const parts = (float*)((char*)workspace + 256 + sh.spans);
  const auto kernel = attn_step_kernel<IT, DP, Engine>;
  const size_t smem = step_smem<IT, DP>(sh.d.G < kHeads ? sh.d.G : kHeads);
  cudaError_t e = set_smem_once((const void*)kernel, step_smem<IT, DP>(kHeads));
  if (e != cudaSuccess) return e;
  StepMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (sh.d.num_pages > 0) {  // without pages no copy is issued
    const bool bf16 = sizeof(IT) == 2;
    const uint64_t dims[4] = {(uint64_t)sh.d.D, (uint64_t)sh.d.Hk, (uint64_t)sh.d.page_size, (uint64_t)sh.d.num_pages};
    const uint32_t box[4] = {(uint32_t)slab_features<IT>(), 1, (uint32_t)sh.d.box, 1};
    if (!get_encoder() || !map_4d(&maps.k, kc, bf16, dims, box) || !map_4d(&maps.v, vc, bf16, dims, box)) return cudaErrorInvalidValue;
  }
  e = attn_launch(kernel, sh.blocks, kThreads + 32, smem, 1, s, maps, sh.d, (const IT*)q, (const IT*)k, (const IT*)v, (IT*)kc, (IT*)vc, table,
                  lengths, (IT*)o, spans, parts, status);
  if (e != cudaSuccess) return e;
  stage_mark(s, "attn_step");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Where units are few each is in many parts: 20 loads a warp instead of 8, which keep more registers than many small joins can spare.
  const auto join = (long long)sh.blocks >= 32ll * sh.d.B * sh.d.Hk * sh.d.HB ? attn_join_kernel<IT, DP, 20> : attn_join_kernel<IT, DP, 8>;
  e = attn_launch(join, (long long)sh.d.B * sh.d.Hq, kThreads, 0, 1, s, sh.d, lengths, (IT*)o, (const int2*)spans, (const float*)parts);
  if (e != cudaSuccess) return e;
  stage_mark(s, "attn_join");
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_attn_step_workspace_bytes(const gdr_cache_problem* p) {
  return check_cache(p, true) == GDR_OK ? step_shape(p).bytes : 0;
}

gdr_status gdr_attn_step(const gdr_cache_problem* p, const void* q, const void* k, const void* v, void* k_cache,
                         void* v_cache, const int32_t* block_table, const int32_t* lengths, void* o, void* workspace,
                         size_t workspace_bytes, gdr_stream_t stream) {
  const gdr_status st = check_cache(p, true);
  if (st != GDR_OK) return st;
  if (p->B == 0) return GDR_OK;
  if (!q || !k || !v || !lengths || !o || (p->num_pages > 0 && (!k_cache || !v_cache)) || (p->max_pages > 0 && !block_table))
    return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(q, el) || !elem_ok(k, el) || !elem_ok(v, el) || !elem_ok(o, el) || !elem_ok(block_table, 4) || !elem_ok(lengths, 4) ||
      !vec_ok(k_cache) || !vec_ok(v_cache))
    return GDR_ERR_ALIGNMENT;
  StepShape sh = step_shape(p);
  if (!workspace || workspace_bytes < sh.bytes) return GDR_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return GDR_ERR_ALIGNMENT;
  sh.d.vec = vec_ok(q) && vec_ok(k) && vec_ok(v) && sh.d.ld_q * el % 16 == 0 && sh.d.ld_k * el % 16 == 0 && sh.d.ld_v * el % 16 == 0;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  auto run = [&](auto it, auto dp, auto engine) {
    return status_of(step<decltype(it), decltype(dp)::value, typename decltype(engine)::type>(sh, q, k, v, k_cache, v_cache, block_table, lengths,
                                                                                              o, workspace, s));
  };
  using W = std::integral_constant<int, 128>;
  using N = std::integral_constant<int, 64>;
  const bool wide = p->D > 64, few = sh.d.G <= 4;
  if (p->dtype == GDR_DTYPE_BF16)
    return wide ? run(__nv_bfloat16{}, W{}, std::common_type<EngineBf16<128>>{}) : run(__nv_bfloat16{}, N{}, std::common_type<EngineBf16<64>>{});
  if (wide) return few ? run(0.f, W{}, std::common_type<EngineF32<128, 4>>{}) : run(0.f, W{}, std::common_type<EngineF32<128, kHeads>>{});
  return few ? run(0.f, N{}, std::common_type<EngineF32<64, 4>>{}) : run(0.f, N{}, std::common_type<EngineF32<64, kHeads>>{});
}

size_t gdr_cache_write_workspace_bytes(const gdr_cache_problem* p) { return check_cache(p, false) == GDR_OK && p->cu_seqlens ? 256 : 0; }

gdr_status gdr_cache_write(const gdr_cache_problem* p, const void* k, const void* v, void* k_cache, void* v_cache,
                           const int32_t* block_table, const int32_t* starts, void* workspace, size_t workspace_bytes,
                           gdr_stream_t stream) {
  const gdr_status st = check_cache(p, false);
  if (st != GDR_OK) return st;
  const long long wk = (long long)p->Hk * p->D, tokens = p->cu_seqlens ? p->T : (long long)p->B * p->T;
  if (p->cu_seqlens && p->B < 1) return GDR_ERR_INVALID_ARG;
  if (tokens > 0 && (!k || !v || (p->num_pages > 0 && (!k_cache || !v_cache)) || (p->max_pages > 0 && !block_table))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(k, el) || !elem_ok(v, el) || !elem_ok(block_table, 4) || !elem_ok(starts, 4) || !elem_ok(p->cu_seqlens, 4) || !vec_ok(k_cache) ||
      !vec_ok(v_cache) || ((uintptr_t)workspace & 255u))
    return GDR_ERR_ALIGNMENT;
  if (p->cu_seqlens && (!workspace || workspace_bytes < 256)) return GDR_ERR_WORKSPACE;
  const WriteDims d{p->B, p->T, p->Hk, p->D, p->num_pages, p->page_size, p->max_pages, p->cu_seqlens, tokens, p->ld_k ? p->ld_k : wk,
                    p->ld_v ? p->ld_v : wk};
  const int n16 = (int)(16 / el);
  const bool vec = vec_ok(k) && vec_ok(v) && d.ld_k % n16 == 0 && d.ld_v % n16 == 0;
  const long long threads = tokens * ((wk / (vec ? n16 : 1) + kPieces - 1) / kPieces);
  const long long grid = threads == 0 ? (p->cu_seqlens ? 1 : 0) : (threads + 255) / 256;
  if (grid == 0) return GDR_OK;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  auto go = [&](auto it, auto vv) {
    using IT = decltype(it);
    const cudaError_t e = attn_launch(cache_write_kernel<IT, decltype(vv)::value>, grid, 256, 0, 1, s, d, (const IT*)k, (const IT*)v,
                                      (IT*)k_cache, (IT*)v_cache, block_table, starts, (uint32_t*)workspace);
    if (e != cudaSuccess) return status_of(e);
    stage_mark(s, "cache_write");
    return status_of(cudaGetLastError());
  };
  using C1 = std::integral_constant<int, 1>;
  if (p->dtype == GDR_DTYPE_BF16) return vec ? go(__nv_bfloat16{}, std::integral_constant<int, 8>{}) : go(__nv_bfloat16{}, C1{});
  return vec ? go(0.f, std::integral_constant<int, 4>{}) : go(0.f, C1{});
}

}  // extern "C"
