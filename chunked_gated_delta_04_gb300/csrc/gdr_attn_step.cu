// gdr_attn_step.cu -- attention of one token per sequence over a paged cache, and the write of a prompt into it
// (include/gdr_attn.h).
//
// The step reads the visible part of the cache once and is bound by that.  The work is the list of all tiles of 64
// (bf16) or 32 (fp32) positions of all rows and key heads, one behind the other; a launch of two blocks per SM cuts the list into
// equal parts, so that one long sequence, many short ones and any mixture of them load every SM alike.  Which rows have
// how many tiles is on the device only (lengths): every block sums them up itself.  A block takes its tiles in order, with the
// copies of the next two under way (cp.async; a step's rows are 256-byte pieces, wherever their page lies), and keeps
// the running maximum m, sum l and O of a (row, key head), for up to 16 query heads that share it:
//   bf16: mma.m16n8k16, query heads as the rows, so that P's accumulator is the next product's operand; a warp takes 16 of a
//         tile's positions.  The products are small beside the copies (16 rows of 16 positions of 128 features: 32 instructions).
//   fp32: on the FMA pipes, 4 lanes per position for S, 4 features per lane for O.
// A (row, key head) that lies within one block is finished there; of the others each block leaves its part (m, l, O), and a
// second launch adds them in order.  The new token's key and value go from the call's inputs to shared memory and the cache.
#include <cmath>

#include "gdr_attn.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
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
};

// Positions that a tile covers, and the tile of a row's first visible position.
template <typename IT> constexpr int tile_keys() { return sizeof(IT) == 2 ? 64 : 32; }

// The visible positions lo .. len of a row and its tiles; false: the row is skipped.
struct Row {
  int len, lo, tile0, tiles;
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

// Tiles of the rows before thread t's rows (B cut into kThreads runs), and of all: prefix[kThreads + 1] in shared memory.
template <int KT>
__device__ __forceinline__ void sum_rows(const StepDims& d, const int32_t* lengths, long long* prefix) {
  const int tid = threadIdx.x, run = (d.B + kThreads - 1) / kThreads;
  long long sum = 0;
  for (int b = tid * run; b < min(d.B, (tid + 1) * run); ++b) sum += row_of<KT>(d, lengths, b).tiles;
  long long v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if ((tid & 31) >= o) v += y;
  }
  prefix[tid + 1] = v;  // within the warp
  if (tid == 0) prefix[0] = 0;
  __syncthreads();
  long long before = 0;
  for (int w = 0; w < (tid >> 5); ++w) before += prefix[32 * (w + 1)];
  __syncthreads();
  prefix[tid + 1] = v + before;
  __syncthreads();
}

// Where a position of the flat list of tiles lies: row, unit of the row (key head and block of query heads), tile of the unit.
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
    while (rest >= (long long)row.tiles * units) {
      rest -= (long long)row.tiles * units;
      row = row_of<KT>(d, lengths, ++b);
    }
    unit = (int)(rest / row.tiles);
    tile = (int)(rest % row.tiles);
  }
  // The next tile, of which there is one.
  __device__ __forceinline__ void next(const StepDims& d, const int32_t* lengths, int units) {
    if (++tile < row.tiles) return;
    tile = 0;
    if (++unit < units) return;
    unit = 0;
    do row = row_of<KT>(d, lengths, ++b);
    while (row.tiles == 0);
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

// 16 bytes, or zeros (`bytes` 0, nothing is read), past the L1: a cache is read once.
__device__ __forceinline__ void copy_async_l2(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}

// The larger, or a NaN where there is one: it has to reach the row's result.
__device__ __forceinline__ float max_nan(float a, float b) { return b > a || b != b ? b : a; }

// Running softmax of a warp's part of the tiles, products on the tensor cores.
template <int DP>
struct EngineBf16 {
  static constexpr int kRows = kHeads;  // of the accumulator in shared memory
  uint32_t qa[DP / 16][4];
  float O[DP / 8][4], m[2], l[2];  // heads lane / 4 and lane / 4 + 8; m in units of S

  __device__ __forceinline__ void begin(const __nv_bfloat16* q, int heads, const StepDims& d) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = g + 8 * (i & 1), f = 16 * kk + c + 8 * (i >> 1);
        uint32_t w = 0;
        if (r < heads && f < d.D) {  // D is even
          const __nv_bfloat16* at = q + (long long)r * d.D + f;
          const __nv_bfloat162 two = __halves2bfloat162(at[0], at[1]);
          w = *reinterpret_cast<const uint32_t*>(&two);
        }
        qa[kk][i] = w;
      }
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[n][i] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // The warp's 16 positions of a tile whose first position is p0: K and V rows of DP + 8 elements.
  __device__ __forceinline__ void tile(const __nv_bfloat16* K, const __nv_bfloat16* V, int p0, const Row& row, float c, int) {
    constexpr int S = DP + 8;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t ka = smem_addr(K) + 2 * ((16 * w + (lane & 7) + 8 * (lane >> 4)) * S + 8 * (lane >> 3 & 1));
    float s[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      uint32_t b[4];
      ldmatrix4(b, ka + 32 * kk);
      mma16816(s[0], qa[kk], b[0], b[1]);
      mma16816(s[1], qa[kk], b[2], b[3]);
    }
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
      const float base = top[r] == -INFINITY ? 0.f : top[r] * c, f = ex2f(fmaf(m[r], c, -base));
      m[r] = top[r];
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0_ = ex2f(fmaf(s[n][2 * r], c, -base)), p1_ = ex2f(fmaf(s[n][2 * r + 1], c, -base));
        sum += p0_ + p1_;
        pa[2 * n + r] = pack_bf16(p0_, p1_);
      }
      l[r] = fmaf(l[r], f, sum);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        O[n][2 * r] *= f;
        O[n][2 * r + 1] *= f;
      }
    }
    const uint32_t va = smem_addr(V) + 2 * ((16 * w + (lane & 15)) * S + 8 * (lane >> 4));
#pragma unroll
    for (int n = 0; n < DP / 16; ++n) {
      uint32_t b[4];
      ldmatrix4t(b, va + 32 * n);
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
  // acc[head][feature] = (first ? 0 : acc) + O f(head).
  template <typename F>
  __device__ __forceinline__ void add(float* acc, bool first, int, F f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int head = (lane >> 2) + 8 * r;
      const float by = f(head);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        float2* at = reinterpret_cast<float2*>(acc + head * DP + 8 * n + 2 * (lane & 3));
        float2 v = first ? make_float2(0.f, 0.f) : *at;
        v.x = fmaf(O[n][2 * r], by, v.x);
        v.y = fmaf(O[n][2 * r + 1], by, v.y);
        *at = v;
      }
    }
  }
};

// The same in fp32; NH: query heads that it is built for (at least the unit's).
template <int DP, int NH>
struct EngineF32 {
  static constexpr int kRows = NH;
  static constexpr int F = DP / 32;  // features of O per lane: F lane ..
  const float* q;                    // shared memory [NH][DP], zeros behind the heads and features
  float O[NH][F], m[NH], l[NH];

  __device__ __forceinline__ void begin(const float* from, int, const StepDims&) {
    q = from;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
#pragma unroll
      for (int i = 0; i < F; ++i) O[r][i] = 0.f;
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
  }
  // The warp's 8 positions of a tile: K and V rows of DP + 4 elements.
  __device__ __forceinline__ void tile(const float* K, const float* V, int p0, const Row& row, float c, int) {
    constexpr int S = DP + 4;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const float* kr = K + (8 * w + (lane >> 2)) * S;
    float s[NH];
#pragma unroll
    for (int r = 0; r < NH; ++r) s[r] = 0.f;
#pragma unroll
    for (int k = 0; k < DP; k += 16) {
      const float4 a = *reinterpret_cast<const float4*>(kr + k + 4 * (lane & 3));
#pragma unroll
      for (int r = 0; r < NH; ++r) {
        const float4 b = *reinterpret_cast<const float4*>(q + r * DP + k + 4 * (lane & 3));
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
      const float base = top == -INFINITY ? 0.f : top * c, f = ex2f(fmaf(m[r], c, -base));
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
      for (int i = 0; i < F; ++i) v[i] = V[(8 * w + j) * S + F * lane + i];
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
  __device__ __forceinline__ void add(float* acc, bool first, int, Fn f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < NH; ++r) {
      const float by = f(r);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        float* at = acc + r * DP + F * lane + i;
        *at = fmaf(O[r][i], by, first ? 0.f : *at);
      }
    }
  }
};

template <typename IT, int DP>
constexpr int row_elements() { return DP + 16 / (int)sizeof(IT); }
template <typename IT, int DP>
constexpr size_t stage_bytes() { return 2 * sizeof(IT) * tile_keys<IT>() * row_elements<IT, DP>(); }
template <typename IT, int DP>  // the stages, the accumulator, fp32: the queries
constexpr size_t step_smem(int rows) {
  return kStages * stage_bytes<IT, DP>() + sizeof(float) * rows * DP * (sizeof(IT) == 4 ? 2 : 1);
}
// A part: O [kHeads][DP], m [kHeads], l [kHeads] (l < 0: the row needs a page outside the pool).
template <int DP>
constexpr int part_floats() { return kHeads * (DP + 2); }

template <typename IT, int DP, typename Engine>
__global__ void __launch_bounds__(kThreads) attn_step_kernel(StepDims d, const IT* __restrict__ q, const IT* __restrict__ k,
                                                             const IT* __restrict__ v, IT* __restrict__ k_cache, IT* __restrict__ v_cache,
                                                             const int32_t* __restrict__ table, const int32_t* __restrict__ lengths,
                                                             IT* __restrict__ o, float* __restrict__ parts) {
  constexpr int KT = tile_keys<IT>(), S = row_elements<IT, DP>(), N = 16 / (int)sizeof(IT);
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ long long prefix[kThreads + 1];
  __shared__ float ms[kWarps][kHeads], ls[kWarps][kHeads];
  IT* const stages = reinterpret_cast<IT*>(smem);
  float* const acc = reinterpret_cast<float*>(smem + kStages * stage_bytes<IT, DP>());
  const int tid = threadIdx.x, warp = tid >> 5, units = d.Hk * d.HB;
  sum_rows<KT>(d, lengths, prefix);
  const long long total = prefix[kThreads] * units;
  const long long blocks = min((long long)gridDim.x, total);  // that have a tile
  if (blockIdx.x >= blocks) return;
  const long long start = total * blockIdx.x / blocks, end = total * (blockIdx.x + 1) / blocks;

  constexpr int TPR = DP / N, RP = kThreads / TPR, PASS = KT / RP;  // threads of a row, rows at a time, rows of a thread
  const int c_of = tid % TPR * N, r_of = tid / TPR;
  // The pages of the thread's rows of a tile: -1 for a position that is not seen, -2 for a page outside the pool.
  auto pages_of = [&](const Cursor<KT>& from, int (&pages)[PASS]) {
    const int p0 = (from.row.tile0 + from.tile) * KT, first = p0 / d.page_size, rest = p0 - first * d.page_size;
    const int32_t* at = table + (long long)from.b * d.max_pages + first;
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int r = r_of + RP * i, x = rest + r;
      const bool seen = p0 + r >= from.row.lo && p0 + r <= from.row.len;
      pages[i] = seen ? at[d.page_size >= KT ? (int)(x >= d.page_size) : x / d.page_size] : -1;
      if (seen && (pages[i] < 0 || pages[i] >= d.num_pages)) pages[i] = -2;
    }
  };
  // The copies of the tile at `from` into a stage; true: a page outside the pool.
  auto load = [&](const Cursor<KT>& from, const int (&pages)[PASS], int stage) {
    IT* const ks = stages + (size_t)stage * 2 * KT * S + r_of * S + c_of;
    IT* const vs = ks + KT * S;
    const int h = from.unit / d.HB, p0 = (from.row.tile0 + from.tile) * KT, rest = p0 % d.page_size;
    const int last = from.row.len - p0;  // the new token's row, if it is one of the tile's
    const bool wide = c_of < d.D;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      const int r = r_of + RP * i, x = rest + r;
      const int place = d.page_size >= KT ? (x >= d.page_size ? x - d.page_size : x) : x % d.page_size;
      const bool ok = pages[i] >= 0 && wide;
      bad |= pages[i] == -2;
      const long long at = ok ? (((long long)pages[i] * d.page_size + place) * d.Hk + h) * d.D + c_of : 0;
      if (r != last) {
        copy_async_l2(ks + RP * i * S, k_cache + at, ok ? 16 : 0);
        copy_async_l2(vs + RP * i * S, v_cache + at, ok ? 16 : 0);
        continue;
      }
      uint4 kn = make_uint4(0, 0, 0, 0), vn = kn;
      if (wide) {
        const IT *kf = k + (long long)from.b * d.ld_k + (long long)h * d.D + c_of, *vf = v + (long long)from.b * d.ld_v + (long long)h * d.D + c_of;
        if (d.vec) {
          kn = *reinterpret_cast<const uint4*>(kf);
          vn = *reinterpret_cast<const uint4*>(vf);
        } else {
          alignas(16) IT a[N], b[N];
#pragma unroll
          for (int e = 0; e < N; ++e) a[e] = kf[e], b[e] = vf[e];
          kn = *reinterpret_cast<const uint4*>(a);
          vn = *reinterpret_cast<const uint4*>(b);
        }
      }
      *reinterpret_cast<uint4*>(ks + RP * i * S) = kn;
      *reinterpret_cast<uint4*>(vs + RP * i * S) = vn;
      if (ok && from.unit % d.HB == 0) {  // one unit of a key head writes
        *reinterpret_cast<uint4*>(k_cache + at) = kn;
        *reinterpret_cast<uint4*>(v_cache + at) = vn;
      }
    }
    return bad;
  };

  Cursor<KT> here, ahead;
  here.seek(d, lengths, prefix, units, start);
  ahead = here;
  uint32_t bad_stages = 0;
  long long loaded = start;
  int pages[PASS];  // of the tile whose copies are next: read a tile ahead of them
  pages_of(ahead, pages);
  auto load_next = [&](int into) {
    bad_stages &= ~(1u << into);
    if (loaded < end) {
      bad_stages |= (uint32_t)load(ahead, pages, into) << into;
      if (++loaded < end) {
        ahead.next(d, lengths, units);
        pages_of(ahead, pages);
      }
    }
    copy_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load_next(i);
  Engine e;
  const float c = d.scale * kLog2e;
  int stage = 0, first_tile = here.tile, heads = 0;
  bool fresh = true, bad = false;
  for (long long at = start; at < end; ++at) {
    if (fresh) {
      const int hb = here.unit % d.HB, h0 = here.unit / d.HB * d.G + hb * kHeads;
      heads = min(kHeads, d.G - hb * kHeads);
      const IT* from = q + (long long)here.b * d.ld_q + (long long)h0 * d.D;
      if constexpr (sizeof(IT) == 4) {
        float* qs = acc + Engine::kRows * DP;
        for (int i = tid; i < Engine::kRows * DP; i += kThreads) qs[i] = i / DP < heads && i % DP < d.D ? from[(long long)(i / DP) * d.D + i % DP] : 0.f;
        e.begin(qs, heads, d);  // the barrier below orders it
      } else {
        e.begin(from, heads, d);
      }
      first_tile = here.tile;
      fresh = bad = false;
    }
    copy_async_wait_group<kStages - 2>();
    __syncthreads();
    load_next((stage + kStages - 1) % kStages);
    const IT* ks = stages + (size_t)stage * 2 * KT * S;
    e.tile(ks, ks + KT * S, (here.row.tile0 + here.tile) * KT, here.row, c, heads);
    bad |= bad_stages >> stage & 1;
    stage = (stage + 1) % kStages;
    if (here.tile + 1 < here.row.tiles && at + 1 < end) {
      ++here.tile;
      continue;
    }
    // the end of a (row, unit), or of the block's part of it
    e.stats(ms[warp], ls[warp], heads);
    bad = __syncthreads_or(bad);
    auto top_of = [&](int r) { return max_nan(max_nan(ms[0][r], ms[1][r]), max_nan(ms[2][r], ms[3][r])); };
    auto share = [&](int w, int r) {  // of warp w's part in the whole
      const float top = top_of(r), base = top == -INFINITY ? 0.f : top * c;
      return ex2f(fmaf(ms[w][r], c, -base));
    };
    for (int w = 0; w < kWarps; ++w) {
      if (warp == w) e.add(acc, w == 0, heads, [&](int r) { return r < heads ? share(w, r) : 0.f; });
      __syncthreads();
    }
    const bool whole = first_tile == 0 && here.tile + 1 == here.row.tiles;
    float* const part = parts + ((long long)blockIdx.x * 2 + (at - (here.tile - first_tile) > start ? 1 : 0)) * part_floats<DP>();
    for (int i = tid; i < heads * DP; i += kThreads) {
      const int r = i / DP, f = i % DP;
      if (whole) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum = fmaf(ls[w][r], share(w, r), sum);
        const int h = here.unit / d.HB * d.G + here.unit % d.HB * kHeads + r;
        if (f < d.D) o[((long long)here.b * d.Hq + h) * d.D + f] = from_f32<IT>(bad ? 0.f : acc[i] / sum);
      } else {
        part[i] = acc[i];
        if (f == 0) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum = fmaf(ls[w][r], share(w, r), sum);
          part[kHeads * DP + r] = top_of(r);
          part[kHeads * (DP + 1) + r] = bad ? -1.f : sum;
        }
      }
    }
    fresh = true;
    if (at + 1 < end) {
      here.next(d, lengths, units);
      __syncthreads();  // acc, ms and ls are used again
    }
  }
  copy_async_wait();
}

// The rows' results that several blocks have parts of, and zeros for the rows that were skipped.  A block per query head of a row.
template <typename IT, int DP>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(StepDims d, int launched, const int32_t* __restrict__ lengths, IT* __restrict__ o,
                                                             const float* __restrict__ parts) {
  constexpr int KT = tile_keys<IT>();
  __shared__ long long prefix[kThreads + 1];
  __shared__ float red[kWarps][2];
  __shared__ float weight[kThreads];
  const int tid = threadIdx.x, b = (int)(blockIdx.x / (unsigned)d.Hq), h = (int)(blockIdx.x % (unsigned)d.Hq), units = d.Hk * d.HB;
  const Row row = row_of<KT>(d, lengths, b);
  IT* out = o + ((long long)b * d.Hq + h) * d.D;
  if (row.tiles == 0) {
    if (tid < d.D) out[tid] = from_f32<IT>(0.f);
    return;
  }
  sum_rows<KT>(d, lengths, prefix);
  const long long total = prefix[kThreads] * units;
  const int run = (d.B + kThreads - 1) / kThreads;
  const long long blocks = min((long long)launched, total);
  long long before = prefix[b / run];
  for (int x = b / run * run; x < b; ++x) before += row_of<KT>(d, lengths, x).tiles;
  const int unit = h / d.G * d.HB + h % d.G / kHeads, r = h % d.G % kHeads;
  const long long a = before * units + (long long)unit * row.tiles, z = a + row.tiles - 1;
  auto start_of = [&](long long x) { return total * x / blocks; };
  auto block_of = [&](long long at) {
    long long x = at * blocks / total;
    while (start_of(x + 1) <= at) ++x;
    while (start_of(x) > at) --x;
    return (int)x;
  };
  const int c0 = block_of(a), c1 = block_of(z);
  if (c0 == c1) return;
  auto part_of = [&](int x) { return parts + ((long long)x * 2 + (a > start_of(x) ? 1 : 0)) * part_floats<DP>(); };
  const float c = d.scale * kLog2e;
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
  const float base = top == -INFINITY ? 0.f : top * c;
  float sum = 0.f, l = 0.f;
  for (int x0 = c0; x0 <= c1; x0 += kThreads) {  // in order, a hundred parts at a time
    __syncthreads();
    const int n = min(kThreads, c1 - x0 + 1);
    if (tid < n) weight[tid] = ex2f(fmaf(part_of(x0 + tid)[kHeads * DP + r], c, -base));
    __syncthreads();
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float* p = part_of(x0 + i);
      l = fmaf(p[kHeads * (DP + 1) + r], weight[i], l);
      if (tid < DP) sum = fmaf(p[r * DP + tid], weight[i], sum);
    }
  }
  if (tid < d.D) out[tid] = from_f32<IT>(bad > 0.f ? 0.f : sum / l);
}

// ------------------------------------------------------------------------------ prompts to pages
// A copy, bound by memory: 16 bytes of one token and head per thread, k and v one after the other.
struct WriteDims {
  int B, T, Hk, D, num_pages, page_size, max_pages;
  const int32_t* cu;
  long long tokens, ld_k, ld_v;
};

template <typename IT, int V>
__global__ void __launch_bounds__(256) cache_write_kernel(WriteDims d, const IT* __restrict__ k, const IT* __restrict__ v,
                                                          IT* __restrict__ k_cache, IT* __restrict__ v_cache,
                                                          const int32_t* __restrict__ table, const int32_t* __restrict__ starts,
                                                          uint32_t* __restrict__ status) {
  if (d.cu) {
    bool bad = false;
    for (int n = threadIdx.x; n < d.B; n += 256) bad |= d.cu[n] > d.cu[n + 1];
    if (threadIdx.x == 0) bad |= d.cu[0] != 0 || d.cu[d.B] != d.T;
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = bad ? kDevErrBadCuSeqlens : 0u;
    if (bad) return;
  }
  const int wide = d.Hk * d.D / V;
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x, token = x / wide;
  if (token >= d.tokens) return;
  const int c = (int)(x - token * wide) * V;
  const int n = d.cu ? seq_of(d.cu, d.B, token) : (int)(token / d.T);
  const long long t = d.cu ? token - d.cu[n] : token - (long long)n * d.T;
  const long long pos = t + (starts ? starts[n] : 0);
  if (pos < 0 || pos >= (long long)d.max_pages * d.page_size) return;
  const int pi = (int)(pos / d.page_size), page = table[(long long)n * d.max_pages + pi];
  if (page < 0 || page >= d.num_pages) return;
  const long long to = ((long long)page * d.page_size + (pos - (long long)pi * d.page_size)) * d.Hk * d.D + c;
  if constexpr (V == 1) {
    k_cache[to] = k[token * d.ld_k + c];
    v_cache[to] = v[token * d.ld_v + c];
  } else {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(k + token * d.ld_k + c)), b = __ldcs(reinterpret_cast<const uint4*>(v + token * d.ld_v + c));
    *reinterpret_cast<uint4*>(k_cache + to) = a;
    *reinterpret_cast<uint4*>(v_cache + to) = b;
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
  if ((long long)p->max_pages * p->page_size >= most || wk >= most) return GDR_ERR_UNSUPPORTED;
  if (step && (long long)p->B * p->Hq >= most) return GDR_ERR_UNSUPPORTED;
  if (!step && (p->cu_seqlens ? (long long)p->T : (long long)p->B * p->T) >= most) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

struct StepShape {
  StepDims d;
  int blocks;
  size_t bytes;
};
StepShape step_shape(const gdr_cache_problem* p) {
  StepShape s;
  const long long wq = (long long)p->Hq * p->D, wk = (long long)p->Hk * p->D;
  const int G = p->Hq / p->Hk, KT = p->dtype == GDR_DTYPE_BF16 ? tile_keys<__nv_bfloat16>() : tile_keys<float>();
  s.d = StepDims{p->B, p->Hq, p->Hk, p->D, G, (G + kHeads - 1) / kHeads, p->num_pages, p->page_size, p->max_pages, p->window,
                 p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)p->D)), p->ld_q ? p->ld_q : wq, p->ld_k ? p->ld_k : wk,
                 p->ld_v ? p->ld_v : wk, 0};
  const long long most = ((long long)p->max_pages * p->page_size + KT - 1) / KT;  // tiles of a row at most
  const double tiles = (double)p->B * p->Hk * s.d.HB * (double)most;
  s.blocks = tiles < 2 * kSmCount ? (int)tiles : 2 * kSmCount;
  if (s.blocks < 1) s.blocks = 1;
  s.bytes = block_align(sizeof(float) * 2 * (size_t)s.blocks * (p->D > 64 ? part_floats<128>() : part_floats<64>()));
  return s;
}

template <typename IT, int DP, typename Engine>
cudaError_t step(const StepShape& sh, const void* q, const void* k, const void* v, void* kc, void* vc, const int32_t* table,
                 const int32_t* lengths, void* o, float* parts, cudaStream_t s) {
  const auto kernel = attn_step_kernel<IT, DP, Engine>;
  constexpr size_t smem = step_smem<IT, DP>(Engine::kRows);
  cudaError_t e = set_smem_once((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<sh.blocks, kThreads, smem, s>>>(sh.d, (const IT*)q, (const IT*)k, (const IT*)v, (IT*)kc, (IT*)vc, table, lengths, (IT*)o, parts);
  stage_mark(s, "attn_step");
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attn_join_kernel<IT, DP><<<(unsigned)(sh.d.B * sh.d.Hq), kThreads, 0, s>>>(sh.d, sh.blocks, lengths, (IT*)o, parts);
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
  sh.d.vec = vec_ok(k) && vec_ok(v) && sh.d.ld_k * el % 16 == 0 && sh.d.ld_v * el % 16 == 0;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  float* parts = (float*)workspace;
  auto run = [&](auto it, auto dp, auto engine) {
    return status_of(step<decltype(it), decltype(dp)::value, typename decltype(engine)::type>(sh, q, k, v, k_cache, v_cache, block_table, lengths,
                                                                                              o, parts, s));
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
  const long long threads = tokens * (wk / (vec ? n16 : 1));
  const long long grid = threads == 0 ? (p->cu_seqlens ? 1 : 0) : (threads + 255) / 256;
  if (grid == 0) return GDR_OK;
  if (grid >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  auto go = [&](auto it, auto vv) {
    using IT = decltype(it);
    cache_write_kernel<IT, decltype(vv)::value><<<(unsigned)grid, 256, 0, s>>>(d, (const IT*)k, (const IT*)v, (IT*)k_cache, (IT*)v_cache,
                                                                               block_table, starts, (uint32_t*)workspace);
    stage_mark(s, "cache_write");
    return status_of(cudaGetLastError());
  };
  using C1 = std::integral_constant<int, 1>;
  if (p->dtype == GDR_DTYPE_BF16) return vec ? go(__nv_bfloat16{}, std::integral_constant<int, 8>{}) : go(__nv_bfloat16{}, C1{});
  return vec ? go(0.f, std::integral_constant<int, 4>{}) : go(0.f, C1{});
}

}  // extern "C"
