// gdr_ssm.cuh -- the selective scan's units of work, shared by its forward and backward.
//
// A sequence is cut into segments of Lseg tokens (a multiple of 16; one segment where the channels
// alone fill the GPU).  A unit is one segment of one sequence; every sequence has at least one, so
// that an empty one still hands its state on.  States are kept for the backward at the start of
// every 16 tokens of a sequence (a tile).
#pragma once

#include <initializer_list>

#include "gdr_block.cuh"

namespace gdr {

constexpr int kTile = 16;
// A log2(e), finite where A is -infinity, so that D = 0 past a sequence's end gives exp(0) = 1 there
// too; a NaN stays one.
__device__ __forceinline__ float decay_rate(float a) {
  const float r = a * kLog2e;
  return r < -3.4e38f ? -3.4e38f : r;
}

struct SsmDims {
  int D, N, G, Dg, T, num_seqs, softplus;
  long long total, ld_x, ld_dt, ld_b, ld_c, ld_dy;
  int vec;  // rows of x, dt, dy and outputs (bit 0), of B and C (bit 1) aligned to four elements
  int Lseg;
  int seq_units, seq_tiles;  // fixed length: units and tiles of a sequence
  long long max_units, max_tiles;
  const int32_t* cu;
  // variable length, in the workspace: {status, number of units}, unit offsets per sequence, units
  const uint32_t* status;
  const int* unit_off;
  const int4* units;  // {seq | first << 30 | last << 31, first token, tokens, first tile}
};

struct SsmUnit {
  int seq, t0, len;
  long long tile0;
  bool first, last;
};

__device__ __forceinline__ bool ssm_bad(const SsmDims& d) { return d.cu && d.status[0] != 0; }
__device__ __forceinline__ long long ssm_unit_count(const SsmDims& d) {
  return d.cu ? (long long)d.status[1] : (long long)d.num_seqs * d.seq_units;
}
__device__ __forceinline__ SsmUnit ssm_unit(const SsmDims& d, long long u) {
  SsmUnit r;
  if (d.cu) {
    const int4 e = d.units[u];
    r.seq = e.x & 0x3fffffff;
    r.first = (e.x >> 30) & 1;
    r.last = (e.x >> 31) & 1;
    r.t0 = e.y;
    r.len = e.z;
    r.tile0 = e.w;
  } else {
    r.seq = (int)(u / d.seq_units);
    const int s = (int)(u - (long long)r.seq * d.seq_units);
    const long long off = (long long)s * d.Lseg;
    r.first = s == 0;
    r.last = s == d.seq_units - 1;
    r.t0 = (int)((long long)r.seq * d.T + off);
    r.len = (int)min((long long)d.Lseg, (long long)d.T - off);
    r.tile0 = (long long)r.seq * d.seq_tiles + off / kTile;
  }
  return r;
}

// Workspace of either direction.  Segments: per unit the state gradient or state at its boundary
// from a zero start (R [units][D][N], turned into the true boundary in place) and the sum of D_t
// ([units][D]).
struct SsmWorkspace {
  uint32_t* status;
  int* unit_off;
  int4* units;
  float* R;
  float* sum_delta;
  float* grads;    // backward: [grid rows][N + 2][D] sums of dA, dDskip, ddt_bias
  float* bc;       // backward: [channel blocks of a group][tokens][G][2 N] sums of dB, dC
  size_t bytes;
};

// SsmDims::vec for a call's pointers (rows: of D channels; bc: of G N states).
int ssm_vec(const SsmDims& d, size_t el, std::initializer_list<const void*> rows, std::initializer_list<const void*> bc);
bool ssm_split(const SsmDims& d);
gdr_status resolve_ssm(const gdr_ssm_problem* p, bool step, SsmDims* d);
SsmWorkspace ssm_workspace(const SsmDims& d, char* base, bool backward);
cudaError_t ssm_launch_index(SsmDims* d, const SsmWorkspace& w, cudaStream_t s);

// Grid rows (units are dealt to them in turn), channel block and blocks of a group of the backward.
int ssm_bwd_channels(int N);
int ssm_bwd_rows(const SsmDims& d);

// The pass over zero-start segments and the scan over their boundaries.  Forward: R[u] becomes the
// state at the start of unit u (from S0); backward: the state gradient at its end (from dS_T).
struct SsmInputs {
  const void *x, *dt, *Bm, *Cm, *dy;
  const float *A, *Dskip, *dt_bias;
};
cudaError_t ssm_launch_boundaries(const SsmDims& d, gdr_dtype dt, const SsmInputs& in, const float* edge,
                                  const SsmWorkspace& w, bool backward, cudaStream_t s);

// Calls f(lanes per channel) for N = 4 * lanes.
template <typename F>
cudaError_t ssm_lanes(int N, F f) {
  switch (N) {
    case 4: return f(std::integral_constant<int, 1>{});
    case 8: return f(std::integral_constant<int, 2>{});
    case 16: return f(std::integral_constant<int, 4>{});
    case 32: return f(std::integral_constant<int, 8>{});
    default: return f(std::integral_constant<int, 16>{});
  }
}

// softplus_f of two values (and, with sig, their sigmoids).
__device__ __forceinline__ f32x2 softplus2(float x, float y, float* sigx, float* sigy) {
  const float u = ex2f(-kLog2e * fabsf(x)), v = ex2f(-kLog2e * fabsf(y));
  const f32x2 uv = pack2(u, v);
  const f32x2 den = add2(uv, pack2(2.f, 2.f));
  const f32x2 s = mul2(uv, pack2(rcpf(lo2(den)), rcpf(hi2(den)))), q = mul2(s, s);
  f32x2 p = pack2(artanh_c(4), artanh_c(4));
#pragma unroll
  for (int i = 3; i >= 0; --i) p = fma2(p, q, pack2(artanh_c(i), artanh_c(i)));
  if (sigx) {
    const float r = rcpf(1.f + u), t = rcpf(1.f + v);
    *sigx = x >= 0.f ? r : u * r;
    *sigy = y >= 0.f ? t : v * t;
  }
  return fma2(add2(s, s), p, pack2(fmaxf(x, 0.f), fmaxf(y, 0.f)));
}

struct alignas(16) Pair2 {
  f32x2 a, b;
};

// Four neighbouring elements of a row as they come from memory, converted where they are used, so
// that the load is not waited for before that.
template <typename IT>
struct Raw4;
template <>
struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void get(float (&o)[4]) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
};
template <>
struct Raw4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void get(float (&o)[4]) const {
    o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xffff0000u);
    o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xffff0000u);
  }
};
// n of the four exist (n <= 0: none); vec: they are aligned to the four elements' size.
template <typename IT>
__device__ __forceinline__ Raw4<IT> load_raw4(const IT* p, int n, bool vec) {
  Raw4<IT> r;
  if (vec && n >= 4) {
    r.v = *reinterpret_cast<const decltype(r.v)*>(p);
  } else if constexpr (sizeof(IT) == 4) {
    r.v = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
  } else {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    const uint32_t a = n > 0 ? q[0] : 0, b = n > 1 ? q[1] : 0, c = n > 2 ? q[2] : 0, e = n > 3 ? q[3] : 0;
    r.v = make_uint2(a | b << 16, c | e << 16);
  }
  return r;
}
template <typename IT>
__device__ __forceinline__ void store4(IT* p, int n, bool vec, const float (&v)[4]) {
  if (vec && n >= 4) {
    if constexpr (sizeof(IT) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(p) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<IT>(v[i]);
  }
}

// NV values in every lane, summed over LANES = 2^k lanes that are OFF apart: each exchange halves
// the values a lane keeps, so it takes about NV exchanges in place of NV log2(LANES).  Lane l (of
// the LANES) ends with the sums of values index(l) .. index(l) + KEEP - 1 in v[0 .. KEEP).
template <int NV, int LANES, int OFF>
struct LaneSums {
  static constexpr int KEEP = NV >= LANES ? NV / LANES : 1;
  __device__ static __forceinline__ int index(int l) {
    int at = 0;
#pragma unroll
    for (int m = NV / 2, b = 1; m >= 1 && b < LANES; m >>= 1, b <<= 1) at += l & b ? m : 0;
    return at;
  }
  __device__ static __forceinline__ bool holds(int l) { return l < NV; }  // once per value
  __device__ static __forceinline__ void run(float* v, int l) {
#pragma unroll
    for (int m = NV / 2, b = 1; b < LANES; m >>= 1, b <<= 1) {
      if (m >= 1) {
        const bool hi = l & b;
#pragma unroll
        for (int i = 0; i < m; ++i) {
          const float send = hi ? v[i] : v[i + m], keep = hi ? v[i + m] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, b * OFF);
        }
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], b * OFF);
      }
    }
  }
};

}  // namespace gdr
