// gdr_attn_tc.cuh -- what the tensor-core kernels of attention share: tensor maps, rings of tiles in shared memory, the
// tiles that end inside a sequence's last block.
#pragma once

#include "gdr_attn.cuh"
#include "tc_common.cuh"

namespace gdr {

// Rows [r0, r0 + 128) of one head of a [tokens, H, D] tensor as DP / 64 slabs of 64 features (128-byte rows, swizzled); features
// from D on and rows behind the last token arrive as zeros.
template <int DP>
constexpr uint32_t attn_tile_bytes() { return (uint32_t)(DP / 64) * kTcBlock * 128; }

template <int DP>
__device__ __forceinline__ void attn_load_tile(unsigned char* dst, const CUtensorMap* map, uint64_t* bar, int head, long long row) {
#pragma unroll
  for (int s = 0; s < DP / 64; ++s) tc::tma_load_3d(dst + s * kTcBlock * 128, map, bar, 64 * s, head, (int)row);
}

// Rows [from, 128) of a tile become zeros (a warp): they belong to another sequence, and what is in them must not reach
// this one's sums, where it would be multiplied by zero.
template <int DP>
__device__ __forceinline__ void attn_clear_rows(unsigned char* tile, int from) {
  const int lane = threadIdx.x & 31;
  for (int s = 0; s < DP / 64; ++s)
    for (int e = from * 8 + lane; e < kTcBlock * 8; e += 32)
      *reinterpret_cast<uint4*>(tile + s * kTcBlock * 128 + e * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  __syncwarp();
}

// A tile of 128 rows in shared memory as an operand: the low word of its matrix descriptor, whose high word is the same for all.
// K-major (rows are M or N): a K step of 16 features is 32 bytes on, a slab of 64 features the next one.  MN-major (rows are K):
// a step of 16 rows is 2 KB on.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart, 128-byte swizzle
constexpr uint32_t kSlabBytes = kTcBlock * 128;
// (In a cluster an address in shared memory has the block's rank above its low 18 bits.)
__device__ __forceinline__ uint32_t desc_kmajor(uint32_t saddr) { return (saddr >> 4 & 0x3FFFu) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mnmajor(uint32_t saddr) { return (saddr >> 4 & 0x3FFFu) | (kSlabBytes >> 4) << 16; }
__device__ __forceinline__ constexpr uint32_t kmajor_step(int kk) { return (uint32_t)(kk >> 2) * (kSlabBytes >> 4) + (uint32_t)(kk & 3) * 2u; }
__device__ __forceinline__ constexpr uint32_t mnmajor_step(int kk) { return (uint32_t)kk * 128u; }

// The MMAs are issued by one lane, but the whole warp runs the code around them, with a warp index that is the same for all lanes by
// construction (attn_warp): addresses and descriptors then stay in uniform registers, where the instruction wants them.  In a
// branch of one lane each MMA first moved its operands there one by one, which took 90 cycles an MMA of 64.
__device__ __forceinline__ int attn_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }
__device__ __forceinline__ uint32_t attn_leader() {  // 1 in one lane of the warp
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void attn_commit(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// D = A B^T over DP features, A and B K-major tiles.
template <int DP>
__device__ __forceinline__ void attn_scores(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t leader) {
  constexpr uint32_t id = tc::idesc_bf16(kTcBlock, kTcBlock, 0, 0);
  a = desc_kmajor(a);
  b = desc_kmajor(b);
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a + kmajor_step(kk)), "r"(b + kmajor_step(kk)), "r"(kDescHi), "r"(id), "r"(kk > 0 ? 1u : 0u), "r"(leader)
        : "memory");
}
// D (+)= A B: A [128 x 128] in TMEM as bf16 (32 columns for its first 64 columns, those of the others begin at column Second),
// B a tile of 128 rows by DP features; K steps From .. To of its 8.
template <int DP, uint32_t Second = 32, int From = 0, int To = kTcBlock / 16>
__device__ __forceinline__ void attn_product(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool accumulate, uint32_t leader) {
  constexpr uint32_t id = tc::idesc_bf16(kTcBlock, DP, 0, 1);
  b = desc_mnmajor(b);
#pragma unroll
  for (int kk = From; kk < To; ++kk)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem + (kk < 4 ? 8u * kk : Second + 8u * (kk - 4))), "r"(b + mnmajor_step(kk)), "r"(kDescHi), "r"(id),
        "r"(accumulate || kk > 0 ? 1u : 0u), "r"(leader)
        : "memory");
}

// mbar_wait by a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool attn_warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status, uint32_t bit) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, status, bit));
}

// Registers per thread from here on, for a warpgroup: what one gives up another may take.
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 columns of this thread's TMEM lane: 64 values as bf16, the even ones in the lower halves.
__device__ __forceinline__ void attn_put64(uint32_t taddr, const float* v) {
  uint32_t r[32];
#pragma unroll
  for (int y = 0; y < 32; ++y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * y], v[2 * y + 1]);
    r[y] = *reinterpret_cast<const uint32_t*>(&b);
  }
  tc::tmem_st32(taddr, r);
}

// A row of an accumulator, DP columns of this thread's TMEM lane from taddr on, times f to out as bf16 (D features; with `any`
// false or f zero the row is zero, whatever the accumulator holds; nothing is written unless `mine`).
template <int DP>
__device__ __forceinline__ void attn_store_row(uint32_t taddr, __nv_bfloat16* out, int D, float f, bool any, bool mine) {
#pragma unroll
  for (int e = 0; e < DP; e += 32) {
    float o[32];
    if (any) {
      tc::tmem_ld32(taddr + e, o);
      tc::tmem_wait_ld();
    }
    if (mine) {
#pragma unroll
      for (int y = 0; y < 32; y += 8) {
        float v[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) v[z] = any && f != 0.f ? o[y + z] * f : 0.f;
        if (e + y < D) store_v<8>(out + e + y, v);
      }
    }
  }
}

// The same of the sum of two accumulators' rows, times f0 and f1, where there are any.
template <int DP>
__device__ __forceinline__ void attn_store_row(uint32_t taddr0, uint32_t taddr1, __nv_bfloat16* out, int D, float f0, float f1, bool any0,
                                               bool any1, bool mine) {
#pragma unroll
  for (int e = 0; e < DP; e += 32) {
    float o0[32], o1[32];
    if (any0) tc::tmem_ld32(taddr0 + e, o0);
    if (any1) tc::tmem_ld32(taddr1 + e, o1);
    tc::tmem_wait_ld();
    if (mine) {
#pragma unroll
      for (int y = 0; y < 32; y += 8) {
        float v[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) v[z] = (any0 && f0 != 0.f ? o0[y + z] * f0 : 0.f) + (any1 && f1 != 0.f ? o1[y + z] * f1 : 0.f);
        if (e + y < D) store_v<8>(out + e + y, v);
      }
    }
  }
}

// A place in a ring of N slots: slot and parity of its use.
template <int N>
struct AttnRing {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Tensor map of a [rows, H, D] bf16 tensor with token stride ld, for attn_load_tile.
inline bool attn_map(CUtensorMap* m, const void* base, int D, int H, long long rows, long long ld) {
  return get_encoder() && map_3d_rows(m, base, (uint64_t)D, (uint64_t)H, (uint64_t)rows, (uint64_t)ld, kTcBlock);
}

// Work item `turn` of a block: items lie by falling work, and the rounds of the grid take them forth and back, so that a block
// that had the largest of one round gets the smallest of the next.  -1: none is left.
// Where there are fewer items than SMs, the blocks of a cluster share one (blocks: n of them); it is their only one.
__device__ __forceinline__ long long attn_item(unsigned turn, unsigned items, unsigned n = 1) {
  const unsigned block = blockIdx.x / n, grid = gridDim.x / n;
  const long long first = (long long)turn * grid;
  const long long x = first + (turn & 1u ? grid - 1 - block : block);
  return x < items ? x : -1;
}

// Blocks that share an item: as many as SMs allow, at most 8, and no more than an item has steps.
inline int attn_sharers(long long items, long long steps) {
  int n = 1;
  while (n < 8 && items * 2 * n <= kSmCount && 2 * n <= steps) n *= 2;
  return n;
}
__device__ __forceinline__ int attn_cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return (int)n;
}
// Columns [c0, c0 + N) of a row of this block's part [128][DP] in shared memory: 16-byte pieces, placed by the row so that rows do not
// meet in a bank.
template <int DP>
__device__ __forceinline__ uint32_t part_at(int row, int piece) {
  return (uint32_t)(row * DP + 4 * ((piece ^ row) & (DP / 4 - 1)));
}
template <int DP, int N>
__device__ __forceinline__ void put_part(float* part, int row, int c0, uint32_t taddr, float f, bool any) {
#pragma unroll
  for (int e = 0; e < N; e += 16) {
    float o[16];
    if (any) {
      tc::tmem_ld16(taddr + e, o);
      tc::tmem_wait_ld();
    }
#pragma unroll
    for (int y = 0; y < 16; y += 4)
      *reinterpret_cast<float4*>(part + part_at<DP>(row, (c0 + e + y) / 4)) =
          any && f != 0.f ? make_float4(o[y] * f, o[y + 1] * f, o[y + 2] * f, o[y + 3] * f) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
// The same of the sum of two accumulators' rows, times f0 and f1.
template <int DP, int N>
__device__ __forceinline__ void put_part(float* part, int row, int c0, uint32_t taddr0, uint32_t taddr1, float f0, float f1, bool any0, bool any1) {
#pragma unroll
  for (int e = 0; e < N; e += 16) {
    float o[16], p[16];
    if (any0) tc::tmem_ld16(taddr0 + e, o);
    if (any1) tc::tmem_ld16(taddr1 + e, p);
    tc::tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 16; ++y) o[y] = (any0 && f0 != 0.f ? o[y] * f0 : 0.f) + (any1 && f1 != 0.f ? p[y] * f1 : 0.f);
#pragma unroll
    for (int y = 0; y < 16; y += 4)
      *reinterpret_cast<float4*>(part + part_at<DP>(row, (c0 + e + y) / 4)) = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
  }
}
// 16 bytes at the same place of another block's shared memory.
__device__ __forceinline__ float4 load_peer4(const float* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(tc::mapa(tc::smem_u32(p), (uint32_t)rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float load_peer(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::mapa(tc::smem_u32(p), (uint32_t)rank)) : "memory");
  return v;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const float x[4] = {v.x, v.y, v.z, v.w};
  store_v<4>(p, x);
}
// This block's share of the rows, summed over the n blocks' parts in the order of their ranks, times f; by 256 threads.
template <int DP>
__device__ __forceinline__ void sum_parts(const float* part, int rank, int n, __nv_bfloat16* out, long long ld, int rows, int D, float f) {
  const int r0 = kTcBlock * rank / n, r1 = min(rows, kTcBlock * (rank + 1) / n);
  for (int e = threadIdx.x; e < (r1 - r0) * (DP / 4); e += 256) {
    const int r = r0 + e / (DP / 4), q = e % (DP / 4);
    if (4 * q >= D) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < n; ++x) {
      const float4 v = load_peer4(part + part_at<DP>(r, q), x);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    store4(out + (long long)r * ld + 4 * q, make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f));
  }
}

}  // namespace gdr
