// gdr_ssm.cuh -- the selective scan's units of work, shared by its forward and backward.
//
// A sequence is cut into segments of Lseg tokens (a multiple of 16; one segment where the channels
// alone fill the GPU).  A unit is one segment of one sequence; every sequence has at least one, so
// that an empty one still hands its state on.  States are kept for the backward at the start of
// every 16 tokens of a sequence (a tile).
#pragma once

#include "gdr_block.cuh"

namespace gdr {

constexpr int kTile = 16;
constexpr float kBig = 3.4e38f;

struct SsmDims {
  int D, N, G, Dg, T, num_seqs, softplus;
  long long total, ld_x, ld_dt, ld_b, ld_c, ld_dy;
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

// Four values (of tokens 4 i .. 4 i + 3) summed over the NL lanes of a channel.  Afterwards lane ln
// holds kKeep of the sums, v[0 .. kKeep), of tokens tok(ln) + 0 .. kKeep - 1; holds(ln) says whether
// it is the one to use them.
template <int NL>
struct LaneSum {
  static constexpr int kKeep = NL >= 4 ? 1 : NL == 2 ? 2 : 4;
  __device__ static __forceinline__ int tok(int ln) { return NL >= 4 ? ln & 3 : NL == 2 ? 2 * (ln & 1) : 0; }
  __device__ static __forceinline__ bool holds(int ln) { return NL <= 4 || ln < 4; }
  __device__ static __forceinline__ void run(float (&v)[4], int ln) {
    if constexpr (NL >= 4) {
      const bool hi = ln & 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float send = hi ? v[i] : v[i + 2], keep = hi ? v[i + 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
      }
      const bool h1 = ln & 1;
      const float send = h1 ? v[0] : v[1], keep = h1 ? v[1] : v[0];
      v[0] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
#pragma unroll
      for (int o = 4; o < NL; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    } else if constexpr (NL == 2) {
      const bool hi = ln & 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float send = hi ? v[i] : v[i + 2], keep = hi ? v[i + 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
      }
    }
  }
};

}  // namespace gdr
