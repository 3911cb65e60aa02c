// gdr_attn.cu -- the entry points of attention over whole sequences (include/gdr_attn.h): checks, workspace,
// the tile tables of packed batches, delta, and the choice between the tensor-core and the SIMT kernels.
#include <cmath>

#include "gdr_attn.cuh"

namespace gdr {
namespace {

// ------------------------------------------------------------------------------ tile tables
// A packed batch's cu_seqlens are checked, and its tiles written by falling work (tiles of a long causal sequence differ by
// its length; what starts last decides when the launch ends).  One block per table: keys or queries, tiles of `size`.  Bound by latency:
// 9 us for 28580 tokens in eight sequences, of which the launch behind it hides its own set-up.
struct TableSpec {
  int2* table;
  long long slots;
  int size;
  int keys;
};
constexpr int kBins = 1024;

__device__ __forceinline__ int tile_work(const AttnDims& d, const AttnSpan& s, const TableSpec& t, int tile) {
  int lo, hi;
  if (t.keys)
    attn_queries(d, s, tile * t.size, min(s.m, (tile + 1) * t.size), &lo, &hi);
  else
    attn_keys(d, s, tile * t.size, min(s.n, (tile + 1) * t.size), &lo, &hi);
  return max(0, hi - lo);
}

constexpr int kSeqsHere = 1024;  // sequences whose bounds fit in shared memory

__global__ void __launch_bounds__(kBins) attn_tiles_kernel(AttnDims d, TableSpec t0, TableSpec t1, uint32_t* status) {
  __shared__ int bin[kBins], warp_sums[kBins / 32];
  __shared__ int32_t cu_q[kSeqsHere + 1], cu_k[kSeqsHere + 1];
  launch_wait();
  launch_next();
  const TableSpec t = blockIdx.x == 0 ? t0 : t1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool here = d.num_seqs <= kSeqsHere;  // else they are read where they lie
  bool bad = false;
  for (int n = tid; n < d.num_seqs; n += kBins) {
    const int q0 = d.cu_q[n], q1 = d.cu_q[n + 1], k0 = d.cu_k[n], k1 = d.cu_k[n + 1];
    bad |= q0 > q1 || k0 > k1 || (n == 0 && (q0 != 0 || k0 != 0)) || (n == d.num_seqs - 1 && (q1 != d.Tq || k1 != d.Tk));
    if (here) {
      cu_q[n] = q0, cu_q[n + 1] = q1;  // (neighbours write the same)
      cu_k[n] = k0, cu_k[n + 1] = k1;
    }
  }
  bin[tid] = 0;
  bad = __syncthreads_or(bad);
  if (tid == 0 && blockIdx.x == 0) *status = bad ? kDevErrBadCuSeqlens : 0u;
  int used = 0;
  if (!bad) {
    AttnDims own = d;
    if (here) own.cu_q = cu_q, own.cu_k = cu_k;
    const int most = t.keys ? d.Tq : d.Tk, shift = max(0, 32 - __clz(most) - 10);  // of a tile's work; to a bin
    // a warp per sequence, a lane per tile: count the tiles of each amount of work ...
    auto each = [&](auto f) {
      for (int n = warp; n < d.num_seqs; n += kBins / 32) {
        const AttnSpan s = attn_span(own, n);
        const int tiles = ((t.keys ? s.m : s.n) + t.size - 1) / t.size;
        for (int i = lane; i < tiles; i += 32) f(n, i, &bin[kBins - 1 - min(kBins - 1, tile_work(own, s, t, i) >> shift)]);
      }
    };
    each([&](int, int, int* b) { atomicAdd(b, 1); });
    __syncthreads();
    // ... then the bins' starts, and every tile to its place (the order within a bin varies, results do not)
    const int v = bin[tid];
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    int all = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) all += y;
    }
    used = __shfl_sync(0xffffffffu, all, 31);
    const int before = __shfl_sync(0xffffffffu, all, max(0, warp - 1));
    bin[tid] = sum - v + (warp ? before : 0);
    __syncthreads();
    each([&](int n, int i, int* b) { t.table[atomicAdd(b, 1)] = make_int2(n, i); });
  }
  for (long long i = used + tid; i < t.slots; i += kBins) t.table[i] = make_int2(-1, 0);
}

// ------------------------------------------------------------------------------------- delta
// delta_i = do_i . o_i: what the sum of p dp over a row comes to, with the o that was stored.  A warp per row of D features.
// Bound by memory: o and do are read once.  2 x 4096 tokens, 16 heads of 128 in bf16, 67 MB: 20 us, set-up and waiting for the launch before
// included (o has just been written, and is on its way from L2 to memory meanwhile).  Two or four rows per thread, blocks of 64, 128 or 1024
// threads, a grid that stays and loads ahead, and divisions in 32 bits were no faster (20 to 42 us).
template <typename IT>
__global__ void __launch_bounds__(256) attn_delta_kernel(AttnDims d, const IT* o, const IT* dout, float* delta, uint32_t* status, bool vec) {
  launch_wait();
  launch_next();
  if (blockIdx.x == 0 && threadIdx.x == 0 && !d.cu_q) *status = 0;  // of a packed batch: the tile table's kernel
  constexpr int V = 16 / sizeof(IT);
  const int lane = threadIdx.x & 31;
  // rows of at most 128 features: 16 (bf16) or 32 (fp32) lanes of 16 bytes
  constexpr int L = 128 / V, R = 32 / L;
  const long long rows = (long long)d.B * d.Tq * d.Hq;
  const long long row = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * R + lane / L;
  float sum = 0.f;
  const long long token = row / d.Hq;
  const int h = (int)(row - token * d.Hq);
  if (row < rows) {
    const IT* a = o + row * d.D;
    const IT* b = dout + token * d.ld_do + (long long)h * d.D;
    const int c = lane % L * V;
    if (c < d.D) {
      alignas(16) IT x[V], y[V];
      if (vec) {
        *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(a + c);
        *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(b + c);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = a[c + i], y[i] = b[c + i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum = fmaf(to_f32(x[i]), to_f32(y[i]), sum);
    }
  }
#pragma unroll
  for (int x = L / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (row < rows && lane % L == 0) {
    const long long b = d.cu_q ? 0 : token / d.Tq;
    delta[(b * d.Hq + h) * d.Tq + (token - b * d.Tq)] = sum;
  }
}

// -------------------------------------------------------------------------------- the host
gdr_status resolve(const gdr_attn_problem* p, AttnDims* d) {
  if (p == nullptr || p->B < 0 || p->Tq < 0 || p->Tk < 0 || p->num_seqs < 0) return GDR_ERR_INVALID_ARG;
  if (p->Hq <= 0 || p->Hk <= 0 || p->D <= 0 || p->Hq % p->Hk != 0) return GDR_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || (p->causal != 0 && p->causal != 1) || p->window < 0 || std::isnan(p->scale)) return GDR_ERR_INVALID_ARG;
  if (std::isinf(p->scale)) return GDR_ERR_INVALID_ARG;
  if ((p->cu_q == nullptr) != (p->cu_k == nullptr)) return GDR_ERR_INVALID_ARG;
  if (p->cu_q ? p->B != 1 || p->num_seqs < 1 : p->num_seqs != p->B) return GDR_ERR_INVALID_ARG;
  const long long wq = (long long)p->Hq * p->D, wk = (long long)p->Hk * p->D;
  if (p->ld_q < 0 || p->ld_k < 0 || p->ld_v < 0 || p->ld_do < 0) return GDR_ERR_INVALID_ARG;
  if ((p->ld_q && p->ld_q < wq) || (p->ld_do && p->ld_do < wq) || (p->ld_k && p->ld_k < wk) || (p->ld_v && p->ld_v < wk))
    return GDR_ERR_INVALID_ARG;
  if (p->D % 16 != 0 || p->D > 128) return GDR_ERR_UNSUPPORTED;
  const long long most = 1ll << 31, tokens = most - 1024;  // (the end of a sequence's last tile is a 32-bit number, too)
  if ((long long)p->B * p->Tq >= tokens || (long long)p->B * p->Tk >= tokens) return GDR_ERR_UNSUPPORTED;
  d->B = p->B, d->Tq = p->Tq, d->Tk = p->Tk, d->Hq = p->Hq, d->Hk = p->Hk, d->D = p->D, d->G = p->Hq / p->Hk;
  d->num_seqs = p->num_seqs, d->cu_q = p->cu_q, d->cu_k = p->cu_k;
  d->causal = p->causal;
  d->window = p->window >= p->Tk ? 0 : p->window;  // a window as wide as the keys hides nothing
  if (d->window && (long long)p->Tq + d->window >= tokens) return GDR_ERR_UNSUPPORTED;  // (where a window begins is such a number, too)
  d->scale = p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)p->D));
  d->ld_q = p->ld_q ? p->ld_q : wq, d->ld_do = p->ld_do ? p->ld_do : wq;
  d->ld_k = p->ld_k ? p->ld_k : wk, d->ld_v = p->ld_v ? p->ld_v : wk;
  // the smallest tiles are the SIMT kernels'
  if (attn_tile_count(*d, false, kSimtTile) * d->Hq >= most || attn_tile_count(*d, true, kSimtTile) * d->Hk >= most)
    return GDR_ERR_UNSUPPORTED;
  if (((long long)d->B * d->Tq * d->Hq + 7) / 8 >= most) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

// Whether TMA can copy rows of a head from there.
bool tma_rows(const void* p, long long ld) { return vec_ok(p) && ld * 2 % 16 == 0; }

// Workspace: the status word, then the tile tables of a packed batch (queries, and for the backward keys), then delta.
// Tables are sized for the smaller tiles, whichever kernels a call's alignment selects.
size_t table_bytes(const AttnDims& d, bool keys) { return d.cu_q ? block_align(sizeof(int2) * attn_tile_count(d, keys, kSimtTile)) : 0; }
size_t delta_bytes(const AttnDims& d) { return block_align(sizeof(float) * (size_t)d.B * d.Tq * d.Hq); }
size_t fwd_bytes(const AttnDims& d) { return 256 + table_bytes(d, false); }
size_t bwd_bytes(const AttnDims& d) { return 256 + table_bytes(d, false) + table_bytes(d, true) + delta_bytes(d); }

AttnTiles tiles_of(const AttnDims& d, const int2* table, bool keys, int size) {
  return AttnTiles{d.cu_q ? table : nullptr, ((keys ? d.Tk : d.Tq) + size - 1) / size, keys};
}

cudaError_t launch_tiles(const AttnDims& d, const TableSpec& a, const TableSpec* b, uint32_t* status, cudaStream_t s) {
  const cudaError_t e = attn_launch(attn_tiles_kernel, b ? 2 : 1, kBins, 0, 1, s, d, a, b ? *b : a, status);
  if (e != cudaSuccess) return e;
  stage_mark(s, "attn_tiles");
  return cudaGetLastError();
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_attn_fwd_workspace_bytes(const gdr_attn_problem* p) {
  AttnDims d;
  return resolve(p, &d) == GDR_OK ? fwd_bytes(d) : 0;
}

size_t gdr_attn_bwd_workspace_bytes(const gdr_attn_problem* p) {
  AttnDims d;
  return resolve(p, &d) == GDR_OK ? bwd_bytes(d) : 0;
}

gdr_status gdr_attn_fwd(const gdr_attn_problem* p, const void* q, const void* k, const void* v, void* o, float* lse,
                        void* workspace, size_t workspace_bytes, gdr_stream_t stream) {
  AttnDims d;
  const gdr_status st = resolve(p, &d);
  if (st != GDR_OK) return st;
  const bool queries = d.B > 0 && d.Tq > 0, keys = d.B > 0 && d.Tk > 0;
  if ((queries && (!q || !o || !lse)) || (keys && (!k || !v))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(q, el) || !elem_ok(k, el) || !elem_ok(v, el) || !elem_ok(o, el) || !elem_ok(lse, 4) || !elem_ok(d.cu_q, 4) || !elem_ok(d.cu_k, 4))
    return GDR_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < fwd_bytes(d)) return GDR_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return GDR_ERR_ALIGNMENT;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  char* at = (char*)workspace;
  uint32_t* status = (uint32_t*)at;
  int2* table = (int2*)(at + 256);
  const bool bf16 = p->dtype == GDR_DTYPE_BF16;
  const bool tc = bf16 && queries && keys && tma_rows(q, d.ld_q) && tma_rows(k, d.ld_k) && tma_rows(v, d.ld_v) && vec_ok(o);
  const int size = tc ? attn_fwd_tc_tile(d) : kSimtTile;
  if (d.cu_q) {
    const TableSpec t{table, attn_tile_count(d, false, size), size, 0};
    const cudaError_t e = launch_tiles(d, t, nullptr, status, s);
    if (e != cudaSuccess) return status_of(e);
  }
  if (!queries) return d.cu_q || d.B == 0 ? GDR_OK : status_of(cudaMemsetAsync(status, 0, 4, s));
  const AttnFwdArgs a{q, k, v, o, lse, status};
  const AttnTiles t = tiles_of(d, table, false, size);
  return status_of(tc ? launch_attn_fwd_tc(d, t, size, a, s) : launch_attn_fwd_simt(d, t, bf16, a, s));
}

gdr_status gdr_attn_bwd(const gdr_attn_problem* p, const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                        size_t workspace_bytes, gdr_stream_t stream) {
  AttnDims d;
  const gdr_status st = resolve(p, &d);
  if (st != GDR_OK) return st;
  const bool queries = d.B > 0 && d.Tq > 0, keys = d.B > 0 && d.Tk > 0;
  if ((queries && (!q || !o || !lse || !dout || !dq)) || (keys && (!k || !v || !dk || !dv))) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  for (const void* t : {q, k, v, o, dout, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!elem_ok(t, el)) return GDR_ERR_ALIGNMENT;
  if (!elem_ok(lse, 4) || !elem_ok(d.cu_q, 4) || !elem_ok(d.cu_k, 4)) return GDR_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < bwd_bytes(d)) return GDR_ERR_WORKSPACE;
  if ((uintptr_t)workspace & 255u) return GDR_ERR_ALIGNMENT;
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  char* at = (char*)workspace;
  uint32_t* status = (uint32_t*)at;
  int2* table_q = (int2*)(at + 256);
  int2* table_k = (int2*)(at + 256 + table_bytes(d, false));
  float* delta = (float*)(at + 256 + table_bytes(d, false) + table_bytes(d, true));
  const bool bf16 = p->dtype == GDR_DTYPE_BF16;
  const bool tc = bf16 && queries && keys && tma_rows(q, d.ld_q) && tma_rows(k, d.ld_k) && tma_rows(v, d.ld_v) && tma_rows(dout, d.ld_do) &&
                  vec_ok(dq) && vec_ok(dk) && vec_ok(dv);
  const int size_q = tc ? kTcBlock : kSimtTile, size_k = size_q;
  cudaError_t e = cudaSuccess;
  if (d.cu_q) {
    const TableSpec tq{table_q, attn_tile_count(d, false, size_q), size_q, 0}, tk{table_k, attn_tile_count(d, true, size_k), size_k, 1};
    e = launch_tiles(d, tq, &tk, status, s);
    if (e != cudaSuccess) return status_of(e);
  }
  if (queries) {
    const long long rows = (long long)d.B * d.Tq * d.Hq;
    const bool vec = vec_ok(o) && vec_ok(dout) && d.ld_do * el % 16 == 0;
    if (bf16)
      e = attn_launch(attn_delta_kernel<__nv_bfloat16>, (rows + 15) / 16, 256, 0, 1, s, d, (const __nv_bfloat16*)o,
                      (const __nv_bfloat16*)dout, delta, status, vec);
    else
      e = attn_launch(attn_delta_kernel<float>, (rows + 7) / 8, 256, 0, 1, s, d, (const float*)o, (const float*)dout, delta, status, vec);
    if (e != cudaSuccess) return status_of(e);
    stage_mark(s, "attn_delta");
    e = cudaGetLastError();
    if (e != cudaSuccess) return status_of(e);
  } else if (!d.cu_q && d.B > 0) {
    e = cudaMemsetAsync(status, 0, 4, s);
    if (e != cudaSuccess) return status_of(e);
  }
  const AttnBwdArgs a{q, k, v, dout, lse, delta, dq, dk, dv, status};
  const AttnTiles tq = tiles_of(d, table_q, false, size_q), tk = tiles_of(d, table_k, true, size_k);
  return status_of(tc ? launch_attn_bwd_tc(d, tq, tk, a, s) : launch_attn_bwd_simt(d, tq, tk, bf16, a, s));
}

}  // extern "C"
