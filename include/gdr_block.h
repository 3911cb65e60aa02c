/*
 * gdr_block.h -- C ABI of the operators that stand around the gated delta rule in a model
 * (same library, libgdr.so; same conventions as gdr.h):
 *
 *   gdr_conv_*   short causal depthwise convolution of a mixer's inputs
 *   gdr_ssm_*    selective state space scan (a second recurrent mixer)
 *   gdr_norm_*   norms before and after a block, with its gate and residual scale
 *   gdr_step     the gated delta rule for one token per sequence
 *
 * each for prompts and training (forward, backward) and, where it carries a state, for single
 * tokens (step).  Conventions beyond those of gdr.h:
 *  - Parameters (weights, biases, A, D, scales) and their gradients are float32; activations
 *    have the problem's dtype (F32 or BF16); arithmetic and every sum run in float32.
 *  - Activations that come in may be row-strided: ld_* is the distance between tokens in
 *    elements, at least the row's width; 0 means contiguous.  What goes out is contiguous.
 *    Base pointers need their element's alignment only, and 16-byte aligned pointers and strides
 *    take the vector path, but for the fp32 tensors of states, which are read and written by
 *    16 bytes and refused (GDR_ERR_ALIGNMENT) unless they are aligned to 16: A, S0, S_T, dS_T,
 *    dS0, h_saved and the pools of gdr_ssm_step and gdr_step.  Workspaces: 256 bytes, as in gdr.h.
 *  - Variable length: as in gdr.h (B = 1, cu_seqlens on the device).  A malformed cu_seqlens is
 *    found on the device: nothing is computed and gdr_workspace_status reports it.
 *  - A step reads and writes its states in place in a pool of num_slots states; slots (device,
 *    int32 [B], NULL: row i uses state i) names each row's.  A row whose slot is negative or not
 *    below num_slots is skipped and its output set to zero.  Two rows of one call must not name
 *    the same slot.  Rows of a call: at most 65535 (gdr_step), 262140 (the others).
 *  - Results are bitwise reproducible: no floating-point atomics.
 */
#ifndef GDR_BLOCK_H_
#define GDR_BLOCK_H_

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- short causal convolution
 *   pre[t, c] = bias[c] + sum_{j < W} w[c, j] X[t - (W - 1) + j, c],   y = silu(pre) or pre,
 * X = the sequence's tokens preceded by W - 1 rows of state (zero if state is NULL). */
typedef struct {
  int B, T, C, W;            /* W in 2..4 */
  int num_seqs;              /* fixed length: = B */
  const int32_t* cu_seqlens; /* device, or NULL */
  gdr_dtype dtype;           /* x, y, state, dy, dx, dstate */
  int silu;                  /* 1: y = silu(pre), 0: y = pre */
  long long ld_x, ld_dy;     /* token strides; 0 = C */
  int num_slots;             /* gdr_conv_step only: states in the pool */
} gdr_conv_problem;

/* Bytes of workspace: 0 where none is needed (NULL may be passed). */
size_t gdr_conv_fwd_workspace_bytes(const gdr_conv_problem* p);
size_t gdr_conv_bwd_workspace_bytes(const gdr_conv_problem* p);

/* x [B, T, C]; w [C, W]; bias [C] or NULL; state [num_seqs, W - 1, C] (oldest row first) or NULL;
 * y [B, T, C]; last [num_seqs, W - 1, C] (nullable: the state after the last token). */
gdr_status gdr_conv_fwd(const gdr_conv_problem* p, const void* x, const float* w, const float* bias,
                        const void* state, void* y, void* last, void* workspace, size_t workspace_bytes,
                        gdr_stream_t stream);

/* dy [B, T, C], dlast (nullable: zero) -> dx, dw [C, W], dbias (nullable), dstate (nullable). */
gdr_status gdr_conv_bwd(const gdr_conv_problem* p, const void* x, const float* w, const float* bias,
                        const void* state, const void* dy, const void* dlast, void* dx, float* dw,
                        float* dbias, void* dstate, void* workspace, size_t workspace_bytes,
                        gdr_stream_t stream);

/* One token for each of p->B rows (p->T is 1): x [B, C] (stride ld_x), pool [num_slots, W - 1, C]
 * updated in place, y [B, C]. */
gdr_status gdr_conv_step(const gdr_conv_problem* p, const void* x, const float* w, const float* bias,
                         void* pool, const int32_t* slots, void* y, gdr_stream_t stream);

/* --------------------------------------------------------------- selective state space scan
 *   D_t = softplus(dt_t + dt_bias) (or dt_t + dt_bias),   h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,
 *   y_t[d] = sum_n C_t[n] h_t[d, n] + Dskip[d] x_t[d];
 * channel d uses B and C of group d / (D / G). */
typedef struct {
  int B, T, D, N, G;         /* N in {4, 8, 16, 32, 64}; D % G == 0 */
  int num_seqs;
  const int32_t* cu_seqlens;
  gdr_dtype dtype;           /* x, dt, Bm, Cm, y and their gradients */
  int dt_softplus;
  long long ld_x, ld_dt, ld_b, ld_c, ld_dy; /* token strides; 0 = contiguous (D, or G * N for b, c) */
  int num_slots;             /* gdr_ssm_step only */
} gdr_ssm_problem;

/* Bytes of the states kept for the backward: one [D, N] float32 state at the START of every 16
 * tokens of a sequence; (B * ceil(T / 16), varlen: T / 16 + num_seqs) states. */
size_t gdr_ssm_saved_bytes(const gdr_ssm_problem* p);
size_t gdr_ssm_fwd_workspace_bytes(const gdr_ssm_problem* p);
size_t gdr_ssm_bwd_workspace_bytes(const gdr_ssm_problem* p);

/* x, dt [B, T, D]; A [D, N]; Bm, Cm [B, T, G, N]; Dskip, dt_bias [D] or NULL; S0 [num_seqs, D, N]
 * float32 or NULL -> y [B, T, D]; S_T [num_seqs, D, N] (nullable); h_saved (nullable: nothing kept). */
gdr_status gdr_ssm_fwd(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                       const void* Cm, const float* Dskip, const float* dt_bias, const float* S0, void* y,
                       float* S_T, float* h_saved, void* workspace, size_t workspace_bytes, gdr_stream_t stream);

/* h_saved as written by gdr_ssm_fwd for the same inputs; dS_T nullable (zero).  All outputs but
 * dDskip, ddt_bias and dS0 (nullable) are required. */
gdr_status gdr_ssm_bwd(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                       const void* Cm, const float* Dskip, const float* dt_bias, const float* h_saved,
                       const void* dy, const float* dS_T, void* dx, void* ddt, float* dA, void* dBm, void* dCm,
                       float* dDskip, float* ddt_bias, float* dS0, void* workspace, size_t workspace_bytes,
                       gdr_stream_t stream);

/* One token for each of p->B rows (p->T is 1): pool [num_slots, D, N] float32 updated in place. */
gdr_status gdr_ssm_step(const gdr_ssm_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* Dskip, const float* dt_bias, float* pool,
                        const int32_t* slots, void* y, gdr_stream_t stream);

/* ------------------------------------------------------------------------------- block norms
 *   u = x;  u *= rstd(u) w_post   (w_post given: norm after the block)
 *           u *= silu(z)          (gate given)
 *           u *= scale            (scale given: residual scale per channel)
 *   r = residual + u              (residual given; r is stored in res_dtype)
 *   y = r rstd(r) w_pre           (w_pre given: norm before the next block, of r as stored)
 * rstd(u) = (mean(u^2) + eps)^(-1/2) over the D channels of a row.  Without a residual and with
 * w_pre, y = x rstd(x) w_pre and nothing else may be given; otherwise r is written. */
typedef struct {
  long long tokens;
  int heads, D;              /* rows = tokens * heads, each D <= 16384 wide */
  gdr_dtype dtype;           /* x, z, y, dx, dz, dy; r and dr too when there is no residual */
  gdr_dtype res_dtype;       /* residual, r, dr, dresidual: dtype, or F32 */
  float eps;                 /* > 0 */
  long long ld_x, ld_gate;   /* token strides of x and z; 0 = heads * D */
} gdr_norm_problem;

gdr_status gdr_norm_fwd(const gdr_norm_problem* p, const void* x, const float* w_post, const void* gate,
                        const float* scale, const void* residual, const float* w_pre, void* r, void* y,
                        gdr_stream_t stream);

size_t gdr_norm_bwd_workspace_bytes(const gdr_norm_problem* p);

/* r: the forward's r (required with w_pre; without a residual the forward's x).  dr (nullable: zero)
 * and dy (with w_pre, and only then) are the gradients of r and y; at least one is given.  has_residual says whether
 * the forward had one.  dresidual (nullable) is written when it had; dw_post, dgate, dscale, dw_pre
 * are required where the forward had their tensors. */
gdr_status gdr_norm_bwd(const gdr_norm_problem* p, const void* x, const float* w_post, const void* gate,
                        const float* scale, const void* r, const float* w_pre, int has_residual, const void* dr,
                        const void* dy, void* dx, void* dgate, void* dresidual, float* dw_post, float* dscale,
                        float* dw_pre, void* workspace, size_t workspace_bytes, gdr_stream_t stream);

/* ------------------------------------------------- the gated delta rule, one token per sequence
 * p as for gdr_fwd with T = 1, B rows and no cu_seqlens; dtype, layout, scale and prologue as there
 * (h_dtype, save_wy, cp_fwd, cp_bwd are not used).  q, k [B, Hk, DK]; v, o [B, Hv, DV];
 * g [B, Hv] float32; beta [B, Hv]; pool [num_slots, Hv, DK, DV] (KV) or [num_slots, Hv, DV, DK] (VK)
 * float32, updated in place. */
gdr_status gdr_step(const gdr_problem* p, const void* q, const void* k, const void* v, const float* g,
                    const void* beta, float* pool, int num_slots, const int32_t* slots, void* o,
                    gdr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_BLOCK_H_ */
