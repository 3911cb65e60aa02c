// gdr_step.cu -- the gated delta rule for one token per sequence (include/gdr_block.h):
//
//   p = S k,   S <- e^g S + beta (v - e^g p) k^T,   o = scale S q = scale (e^g S_old q + beta (v - e^g p) (k.q))
//
// S [DV x DK] in fp32.  Bound by memory: the state is read and written once (8 bytes per element,
// 7 operations), everything else is small beside it.  The rows of S (one per value feature) are
// independent, so a head is cut into slices of value features and each slice stays in the
// registers of its block between the load and the store: p and S q are formed in one sweep, the
// update and the store in another, with one reduction between them.  128 rows, 32 heads of 128 x 128:
// 81 us, 6.65 TB/s, the rate of a plain copy; one row of 16 heads: 3.1 us, the launch and one round trip.
//  - VK (S itself): a warp holds whole rows, a lane 4 key features of each; the sums over key
//    features run over the lanes.
//  - KV (S^T): a lane holds 4 value features of some key rows; the sums run over a thread's rows,
//    then over the threads of a column through shared memory.
// Every block forms the head's q, k (normalised, with the prologue), k.q and gates itself: 128
// threads, one element each.
#include "gdr_block.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
// Value features of a block whose keys fit DKP (64 or 128) features: 16 KB of state either way, eight
// 16-byte loads in flight per thread.
constexpr int slice_of(int DKP) { return 32 * 128 / DKP; }

struct StepDims {
  int Hk, Hv, DK, DV, G, num_slots, prologue;
  float scale;
};

__device__ __forceinline__ float block_sum(float v, float* red) {  // red: 4 floats
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename IT, bool KV, int DKP>
__global__ void __launch_bounds__(kThreads) step_kernel(StepDims d, const IT* __restrict__ q, const IT* __restrict__ k,
                                                        const IT* __restrict__ v, const float* __restrict__ g,
                                                        const IT* __restrict__ beta, float* __restrict__ pool,
                                                        const int32_t* __restrict__ slots, IT* __restrict__ o) {
  constexpr int kSlice = slice_of(DKP);
  constexpr int CQ = kSlice / 4;                // KV: float4 columns of the slice; row groups of 128 / CQ rows
  constexpr int LR = DKP / 4, RP = 32 / LR;     // VK: lanes of a row, rows of a warp at a time
  __shared__ __align__(16) float sk[128], sq[128];
  __shared__ float red[4];
  __shared__ float part[2][4][kSlice];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, h = blockIdx.x % d.Hv, v0 = (blockIdx.x / d.Hv) * kSlice;
  const int nv = min(kSlice, d.DV - v0);
  const long long bh = (long long)b * d.Hv + h;
  const int slot = slots ? slots[b] : b;
  IT* oh = o + bh * d.DV + v0;
  if (slot < 0 || slot >= d.num_slots) {
    if (tid < nv) oh[tid] = from_f32<IT>(0.f);
    return;
  }
  float* S = pool + ((long long)slot * d.Hv + h) * d.DK * d.DV;
  // this thread's part of the slice: 8 float4
  float4 st[8];
  if constexpr (KV) {  // rows (128 / CQ) i + tid / CQ of S^T, value features v0 + 4 (tid % CQ) ..
    const int c = 4 * (tid % CQ);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (kThreads / CQ) * i + tid / CQ;
      st[i] = r < d.DK && c < nv ? __ldcs(reinterpret_cast<const float4*>(S + (long long)r * d.DV + v0 + c))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  } else {  // rows v0 + RP (8 warp + i) + lane / LR of S, key features 4 (lane % LR) ..
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = RP * (8 * warp + i) + lane / LR, c = 4 * (lane % LR);
      st[i] = r < nv && c < d.DK ? __ldcs(reinterpret_cast<const float4*>(S + (long long)(v0 + r) * d.DK + c))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // q, k, their product, the gates
  const long long bk = (long long)b * d.Hk + h / d.G;
  float kv = tid < d.DK ? to_f32(k[bk * d.DK + tid]) : 0.f;
  float qv = tid < d.DK ? to_f32(q[bk * d.DK + tid]) : 0.f;
  float gv = g[bh], bt = to_f32(beta[bh]);
  if (d.prologue & GDR_PROLOGUE_QK_L2NORM) {
    kv *= rsqrtf(block_sum(kv * kv, red) + 1e-6f);
    qv *= rsqrtf(block_sum(qv * qv, red) + 1e-6f);
  }
  if (d.prologue & GDR_PROLOGUE_G_LOGSIGMOID) gv = -softplus_f(-gv, nullptr);
  if (d.prologue & GDR_PROLOGUE_BETA_SIGMOID) bt = sigmoid_f(bt);
  const float eg = expf(gv);
  sk[tid] = kv;
  sq[tid] = qv;
  const float kq = block_sum(kv * qv, red);  // its barriers order sk, sq too

  if constexpr (KV) {
    const int c = 4 * (tid % CQ);
    float p[4] = {}, z[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (kThreads / CQ) * i + tid / CQ;
      const float kr = sk[r], qr = sq[r];
      const float e[4] = {st[i].x, st[i].y, st[i].z, st[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = fmaf(e[j], kr, p[j]);
        z[j] = fmaf(e[j], qr, z[j]);
      }
    }
#pragma unroll
    for (int off = CQ; off < 32; off <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] += __shfl_xor_sync(0xffffffffu, p[j], off);
        z[j] += __shfl_xor_sync(0xffffffffu, z[j], off);
      }
    if (lane < CQ)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        part[0][warp][c + j] = p[j];
        part[1][warp][c + j] = z[j];
      }
    __syncthreads();
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int cc = c + j;
      const float pj = (part[0][0][cc] + part[0][1][cc]) + (part[0][2][cc] + part[0][3][cc]);
      const float zj = (part[1][0][cc] + part[1][1][cc]) + (part[1][2][cc] + part[1][3][cc]);
      const float vv = cc < nv ? to_f32(v[bh * d.DV + v0 + cc]) : 0.f;
      u[j] = bt * fmaf(-eg, pj, vv);
      if (tid < CQ && cc < nv) oh[cc] = from_f32<IT>(d.scale * fmaf(eg, zj, u[j] * kq));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (kThreads / CQ) * i + tid / CQ;
      const float kr = sk[r];
      if (r < d.DK && c < nv)
        __stcs(reinterpret_cast<float4*>(S + (long long)r * d.DV + v0 + c),
               make_float4(fmaf(eg, st[i].x, u[0] * kr), fmaf(eg, st[i].y, u[1] * kr), fmaf(eg, st[i].z, u[2] * kr),
                           fmaf(eg, st[i].w, u[3] * kr)));
    }
  } else {
    const int c = 4 * (lane % LR);
    const float4 k4 = *reinterpret_cast<const float4*>(sk + c), q4 = *reinterpret_cast<const float4*>(sq + c);
    float w[16];  // p of rows 0..7, then S q
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = fmaf(st[i].x, k4.x, fmaf(st[i].y, k4.y, fmaf(st[i].z, k4.z, st[i].w * k4.w)));
      w[8 + i] = fmaf(st[i].x, q4.x, fmaf(st[i].y, q4.y, fmaf(st[i].z, q4.z, st[i].w * q4.w)));
    }
    // 16 sums over the LR lanes of a row: each exchange halves the values a lane keeps, so that lane
    // LR / 16 * i of the row ends with value i (and, of 32 lanes, its neighbour with the other half of it)
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) {
      const int bit = m * LR / 16;
#pragma unroll
      for (int i = 0; i < m; ++i) {
        const bool up = lane & bit;
        const float send = up ? w[i] : w[i + m], keep = up ? w[i + m] : w[i];
        w[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    }
    float total = w[0];
    if constexpr (LR == 32) total += __shfl_xor_sync(0xffffffffu, total, 1);
    const int row0 = lane / LR * LR;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float pi = __shfl_sync(0xffffffffu, total, row0 + LR / 16 * i);
      const float zi = __shfl_sync(0xffffffffu, total, row0 + LR / 16 * (8 + i));
      const int r = RP * (8 * warp + i) + lane / LR;
      const float vv = r < nv ? to_f32(v[bh * d.DV + v0 + r]) : 0.f;
      const float u = bt * fmaf(-eg, pi, vv);
      if (lane % LR == 0 && r < nv) oh[r] = from_f32<IT>(d.scale * fmaf(eg, zi, u * kq));
      if (r < nv && c < d.DK)
        __stcs(reinterpret_cast<float4*>(S + (long long)(v0 + r) * d.DK + c),
               make_float4(fmaf(eg, st[i].x, u * k4.x), fmaf(eg, st[i].y, u * k4.y), fmaf(eg, st[i].z, u * k4.z),
                           fmaf(eg, st[i].w, u * k4.w)));
    }
  }
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" gdr_status gdr_step(const gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                               const void* beta, float* pool, int num_slots, const int32_t* slots, void* o,
                               gdr_stream_t stream) {
  if (p == nullptr || p->T != 1 || p->cu_seqlens || num_slots < 0 || p->B < 0) return GDR_ERR_INVALID_ARG;
  if (p->Hk <= 0 || p->Hv <= 0 || p->DK <= 0 || p->DV <= 0 || p->Hv % p->Hk != 0) return GDR_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || (p->layout != GDR_STATE_KV && p->layout != GDR_STATE_VK)) return GDR_ERR_INVALID_ARG;
  if (p->prologue & ~7u) return GDR_ERR_INVALID_ARG;
  if (p->DK % 16 != 0 || p->DV % 16 != 0 || p->DK > 128 || p->DV > 128) return GDR_ERR_UNSUPPORTED;
  const int DKP = p->DK > 64 ? 128 : 64, slice = slice_of(DKP), slices = (p->DV + slice - 1) / slice;
  if (p->B > 65535 || (long long)p->Hv * slices >= (1ll << 31)) return GDR_ERR_UNSUPPORTED;
  if (p->B == 0) return GDR_OK;
  if (!q || !k || !v || !g || !beta || !o || (!pool && num_slots > 0)) return GDR_ERR_INVALID_ARG;
  const size_t el = dtype_bytes(p->dtype);
  if (!elem_ok(q, el) || !elem_ok(k, el) || !elem_ok(v, el) || !elem_ok(beta, el) || !elem_ok(o, el) ||
      !elem_ok(g, 4) || !elem_ok(slots, 4) || !vec_ok(pool))
    return GDR_ERR_ALIGNMENT;
  StepDims d{p->Hk, p->Hv, p->DK, p->DV, p->Hv / p->Hk, num_slots, (int)p->prologue,
             p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)p->DK))};
  cudaStream_t s = (cudaStream_t)stream;
  stage_begin(s);
  const dim3 grid((unsigned)(p->Hv * slices), (unsigned)p->B);
  auto go = [&](auto it, auto kv) {
    using IT = decltype(it);
    constexpr bool KV = decltype(kv)::value;
    const auto kernel = DKP == 128 ? step_kernel<IT, KV, 128> : step_kernel<IT, KV, 64>;
    kernel<<<grid, kThreads, 0, s>>>(d, (const IT*)q, (const IT*)k, (const IT*)v, g, (const IT*)beta, pool, slots, (IT*)o);
    stage_mark(s, "step");
    return cudaGetLastError();
  };
  const bool kv = p->layout == GDR_STATE_KV;
  if (p->dtype == GDR_DTYPE_BF16)
    return status_of(kv ? go(__nv_bfloat16{}, std::true_type{}) : go(__nv_bfloat16{}, std::false_type{}));
  return status_of(kv ? go(float{}, std::true_type{}) : go(float{}, std::false_type{}));
}
