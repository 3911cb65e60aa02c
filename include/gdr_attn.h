/*
 * gdr_attn.h -- C ABI of the attention mixer that stands beside the gated delta rule in a hybrid
 * model (same library, libgdr.so; same conventions as gdr.h and gdr_block.h):
 *
 *   gdr_rope         rotary positions of queries and keys, and their gradient
 *   gdr_attn_fwd/bwd softmax attention over whole sequences
 *   gdr_attn_step    attention of one token per sequence over a paged cache, which it extends
 *   gdr_cache_write  a prompt's keys and values into such a cache
 *
 *  - Activations have the problem's dtype (F32 or BF16).  Those that come in may be token-strided:
 *    ld_* is the distance between tokens in elements (0: contiguous), the heads of a token being
 *    contiguous.  What goes out is contiguous.  Base pointers need their element's alignment only;
 *    16-byte aligned pointers and strides take the vector and tensor-core paths, but for the pages of
 *    a cache, which are refused (GDR_ERR_ALIGNMENT) unless they are aligned to 16.
 *  - Scores, softmax statistics and every sum are float32.  Products run on the tensor cores for
 *    BF16: the probabilities and the gradients of the scores are rounded to BF16 before the
 *    products that they go into.
 *  - Head sizes D: multiples of 16 up to 128.  Query heads: a multiple of the key heads; query
 *    head h reads key head h / (Hq / Hk).
 *  - Results are bitwise reproducible: no floating-point atomics.
 *  - Values are taken as finite within a sequence: an infinity or NaN in a key or value that a query does
 *    not see may still reach it where both lie in one tile of the sequence.  It never reaches another
 *    sequence or row, nor does what lies in a cache behind a row's end.
 */
#ifndef GDR_ATTN_H_
#define GDR_ATTN_H_

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------------------------------------- rotary positions
 *   y_a = scale (x_a cos t - x_b sin t),   y_b = scale (x_b cos t + x_a sin t),
 *   t = (inverse ? -1 : 1) position * freqs[i],  i < R / 2,
 * for the pairs (a, b) = (i, i + R / 2), or (2i, 2i + 1) if interleaved, of the first R features of
 * every head; features from R on are passed on unchanged.  The gradient is the same map with inverse
 * set.  The angle is reduced exactly (64-bit fixed point in turns): positions of any int32 value. */
typedef struct {
  int B, T, Hq, Hk, D, R;    /* R even, at most D; Hk may be 0 (one tensor); any D up to 1024 */
  int num_seqs;              /* as in gdr.h */
  const int32_t* cu_seqlens; /* device, or NULL; used only without positions */
  gdr_dtype dtype;
  int interleaved, inverse;
  float scale;               /* of the rotated features */
  long long ld_q, ld_k;      /* token strides; 0 = H * D */
} gdr_rope_problem;

/* Bytes of workspace: 256 (a status word) for packed batches without positions, else 0. */
size_t gdr_rope_workspace_bytes(const gdr_rope_problem* p);

/* q [B, T, Hq, D], k [B, T, Hk, D]; freqs [R / 2] float64, radians per position, |freqs| <= 2 pi; positions [B, T] int32,
 * or NULL: a token's place in its sequence.  q_out, k_out may not overlap the inputs. */
gdr_status gdr_rope(const gdr_rope_problem* p, const void* q, const void* k, const double* freqs,
                    const int32_t* positions, void* q_out, void* k_out, void* workspace, size_t workspace_bytes,
                    gdr_stream_t stream);

/* ---------------------------------------------------------------------------------- attention
 *   s_ij = scale q_i . k_j,   p_i = softmax over the visible j,   o_i = sum_j p_ij v_j,   lse_i = log sum_j exp s_ij
 * Of a sequence with n queries and m keys, query i sees key j if  j <= i + m - n  (with causal set)
 * and  j > i + m - n - window  (with window > 0).  A query that sees none has o = 0 and lse = -infinity
 * and no part in the gradients.  Queries, keys, and queries plus a window that is narrower than the keys number fewer than
 * 2^31 - 1024. */
typedef struct {
  int B, Tq, Tk, Hq, Hk, D;
  int num_seqs;              /* fixed length: = B */
  const int32_t* cu_q;       /* device, or NULL; packed batches (B = 1) have both */
  const int32_t* cu_k;
  gdr_dtype dtype;
  int causal, window;        /* window 0: none */
  float scale;               /* not above 0: 1 / sqrt(D) */
  long long ld_q, ld_k, ld_v, ld_do; /* token strides; 0 = H * D */
} gdr_attn_problem;

size_t gdr_attn_fwd_workspace_bytes(const gdr_attn_problem* p);
size_t gdr_attn_bwd_workspace_bytes(const gdr_attn_problem* p);

/* q [B, Tq, Hq, D]; k, v [B, Tk, Hk, D]; o [B, Tq, Hq, D]; lse [B, Hq, Tq] float32. */
gdr_status gdr_attn_fwd(const gdr_attn_problem* p, const void* q, const void* k, const void* v, void* o, float* lse,
                        void* workspace, size_t workspace_bytes, gdr_stream_t stream);

/* o, lse: the forward's (contiguous); dout [B, Tq, Hq, D] -> dq, dk, dv. */
gdr_status gdr_attn_bwd(const gdr_attn_problem* p, const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                        size_t workspace_bytes, gdr_stream_t stream);

/* ------------------------------------------------------------------------------ a paged cache
 * k_cache, v_cache [num_pages, page_size, Hk, D]: pages of page_size positions.  block_table [B, max_pages]
 * int32 names each row's pages in order: position t of row b lies at place t % page_size of page
 * block_table[b][t / page_size].  Two rows of one call must not write to the same place.  Several rows
 * may read the same page.  A table covers fewer than 2^31 - 256 positions. */
typedef struct {
  int B;                     /* rows (gdr_attn_step), sequences (gdr_cache_write) */
  int T;                     /* gdr_cache_write: tokens of a sequence, or all tokens with cu_seqlens; step: 1 */
  int Hq, Hk, D;             /* gdr_cache_write: Hq is not used */
  int num_pages, page_size, max_pages;
  const int32_t* cu_seqlens; /* gdr_cache_write: device [B + 1], or NULL: B sequences of T tokens */
  gdr_dtype dtype;
  int window;                /* gdr_attn_step: 0 or as in gdr_attn_problem */
  float scale;               /* gdr_attn_step: not above 0: 1 / sqrt(D) */
  long long ld_q, ld_k, ld_v; /* token strides; 0 = H * D */
} gdr_cache_problem;

size_t gdr_attn_step_workspace_bytes(const gdr_cache_problem* p);

/* q, o [B, Hq, D]; k, v [B, Hk, D]; lengths [B] int32 (device): the positions that row b's cache holds
 * before the call.  The row's k and v go to position lengths[b], then its query attends to positions
 * 0 .. lengths[b] (with a window, to the last `window` of them).  A row whose length is negative or
 * fills its table is skipped: its output is zero, nothing is written.  One that needs a page outside the
 * pool has an output of zero, too; its k and v are written if their own page is in the pool.  The workspace's
 * status word says whether a wait ran out, after which o is not to be used. */
gdr_status gdr_attn_step(const gdr_cache_problem* p, const void* q, const void* k, const void* v, void* k_cache,
                         void* v_cache, const int32_t* block_table, const int32_t* lengths, void* o, void* workspace,
                         size_t workspace_bytes, gdr_stream_t stream);

/* Bytes of workspace: 256 (a status word) with cu_seqlens, else 0. */
size_t gdr_cache_write_workspace_bytes(const gdr_cache_problem* p);

/* k, v [B, T, Hk, D] (packed: [1, T, Hk, D]); starts [B] int32 (device), or NULL: zero.  Token t of sequence n goes to
 * position starts[n] + t; one whose position is negative or outside the table, or whose page is outside
 * the pool, is left out. */
gdr_status gdr_cache_write(const gdr_cache_problem* p, const void* k, const void* v, void* k_cache, void* v_cache,
                           const int32_t* block_table, const int32_t* starts, void* workspace, size_t workspace_bytes,
                           gdr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_ATTN_H_ */
