// gdr_attn.cuh -- what the kernels of include/gdr_attn.h share: the resolved problem, which keys a
// query sees, and how a block finds its tile.
#pragma once

#include "../../include/gdr_attn.h"
#include "gdr_block.cuh"

namespace gdr {

struct AttnDims {
  int B, Tq, Tk, Hq, Hk, D, G, num_seqs;
  const int32_t* cu_q;  // packed batches, else null
  const int32_t* cu_k;
  int causal, window;   // window: 0, or less than Tk
  float scale;
  long long ld_q, ld_k, ld_v, ld_do;
};

// One sequence: its first query and key among all tokens, how many it has, and where its lse begins
// for head 0 (head h: h * lse_ld further).
struct AttnSpan {
  long long q0, k0, lse0;
  int n, m;
};

__device__ __forceinline__ AttnSpan attn_span(const AttnDims& d, int seq) {
  AttnSpan s;
  if (d.cu_q) {
    s.q0 = d.cu_q[seq];
    s.k0 = d.cu_k[seq];
    s.n = d.cu_q[seq + 1] - (int)s.q0;
    s.m = d.cu_k[seq + 1] - (int)s.k0;
    s.lse0 = s.q0;
  } else {
    s.q0 = (long long)seq * d.Tq;
    s.k0 = (long long)seq * d.Tk;
    s.n = d.Tq;
    s.m = d.Tk;
    s.lse0 = s.q0 * d.Hq;
  }
  return s;
}

// Query i of a sequence sees key j (off = keys - queries).
__device__ __forceinline__ bool attn_sees(const AttnDims& d, int off, int i, int j) {
  return (!d.causal || j <= i + off) && (!d.window || j > i + off - d.window);
}
// Keys [lo, hi) that some of the queries [i0, i1) see (none: lo >= hi).
__device__ __forceinline__ void attn_keys(const AttnDims& d, const AttnSpan& s, int i0, int i1, int* lo, int* hi) {
  const int off = s.m - s.n;
  *lo = d.window ? max(0, i0 + off - d.window + 1) : 0;
  *hi = d.causal ? min(s.m, i1 + off) : s.m;
}
// Queries [lo, hi) that see some of the keys [j0, j1).
__device__ __forceinline__ void attn_queries(const AttnDims& d, const AttnSpan& s, int j0, int j1, int* lo, int* hi) {
  const int off = s.m - s.n;
  *lo = d.causal ? max(0, j0 - off) : 0;
  *hi = d.window ? (int)min((long long)s.n, (long long)j1 - 1 - off + d.window) : s.n;
}

// The running softmax forms probabilities as 2^(s c - base), c = scale log2(e), and a maximum's base is its product with c, rounded.  Sums
// against another maximum are brought to it by the difference of the rounded bases: exactly 1 where the maximum has stayed.  (With
// the product unrounded, in one fma, the factor of every tile is off by the same rounding of it, and older tiles' sums drift with their
// number: by up to 1e-3 after 128 tiles at scores of 200.)
__device__ __forceinline__ float attn_base(float top, float c) { return top == -INFINITY ? 0.f : __fmul_rn(top, c); }
__device__ __forceinline__ float attn_rescale(float m, float c, float base) { return ex2f(__fmul_rn(m, c) - base); }  // of nothing seen: 0

// Tiles of a packed batch: {sequence, tile of it}, those with the most work first; sequence -1 behind the last.
// Fixed length: no table, tiles from the end of a sequence (the most work, if causal) to its start, or, where a tile's work
// falls with its place (keys of a causal problem), from the start on.
struct AttnTiles {
  const int2* table;
  int per_seq;  // fixed length
  int forward;  // fixed length: from the start on
};
// The tile, head and sequence of block `x` of H heads; false: nothing to do.
__device__ __forceinline__ bool attn_tile(const AttnDims& d, const AttnTiles& t, int H, unsigned x, int* seq, int* head, int* tile) {
  *head = (int)(x % (unsigned)H);
  const int y = (int)(x / (unsigned)H);
  if (t.table) {
    const int2 e = t.table[y];
    *seq = e.x;
    *tile = e.y;
    return e.x >= 0;
  }
  *seq = y % d.num_seqs;
  *tile = t.forward ? y / d.num_seqs : t.per_seq - 1 - y / d.num_seqs;
  return true;
}

// Tiles of `size` tokens that a launch covers: of the queries, or of the keys.
inline long long attn_tile_count(const AttnDims& d, bool keys, int size) {
  const long long T = keys ? d.Tk : d.Tq;
  return d.cu_q ? T / size + d.num_seqs : (T + size - 1) / size * d.num_seqs;
}

struct AttnFwdArgs {
  const void *q, *k, *v;
  void* o;
  float* lse;
  uint32_t* status;
};
struct AttnBwdArgs {
  const void *q, *k, *v, *dout;
  const float *lse, *delta;  // delta: like lse
  void *dq, *dk, *dv;
  uint32_t* status;
};

// Launches overlap: one may be set up while the one before it in the stream, of the same call or an earlier one, ends (its blocks get
// their memory and barriers ready), and waits with launch_wait for that one's end before it touches anything but its parameters and its
// own shared memory.  Every kernel here waits, in every block that does anything, so that its end is the end of all before it.
// Operands are not read through __restrict__ pointers or __ldg: such loads may be moved in front of the wait, and take what they read as
// unchanged from the kernel's beginning on.
__device__ __forceinline__ void launch_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;"); }
// 16 bytes that are read once; stays behind launch_wait (volatile).
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
template <typename F, typename... Args>
inline cudaError_t attn_launch(F kernel, long long grid, int threads, size_t smem, int cluster, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[2] = {};
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3((unsigned)grid);
  config.blockDim = dim3((unsigned)threads);
  config.dynamicSmemBytes = smem;
  config.stream = s;
  config.attrs = attr;
  config.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

// SIMT kernels: fp32, and bf16 whose pointers or strides the tensor-core path does not take.
constexpr int kSimtTile = 64;  // queries and keys of a tile
cudaError_t launch_attn_fwd_simt(const AttnDims& d, const AttnTiles& t, bool bf16, const AttnFwdArgs& a, cudaStream_t s);
cudaError_t launch_attn_bwd_simt(const AttnDims& d, const AttnTiles& tq, const AttnTiles& tk, bool bf16, const AttnBwdArgs& a,
                                 cudaStream_t s);

// Tensor-core kernels (bf16): q, k, v, dout aligned for TMA, the outputs for 16-byte stores.
constexpr int kTcBlock = 128;  // rows of an MMA tile: queries, keys
// Queries of a block's work: two tiles side by side, or one (its keys in two lanes) where that leaves SMs without work.
int attn_fwd_tc_tile(const AttnDims& d);
cudaError_t launch_attn_fwd_tc(const AttnDims& d, const AttnTiles& t, int tile, const AttnFwdArgs& a, cudaStream_t s);
cudaError_t launch_attn_bwd_tc(const AttnDims& d, const AttnTiles& tq, const AttnTiles& tk, const AttnBwdArgs& a, cudaStream_t s);

}  // namespace gdr
