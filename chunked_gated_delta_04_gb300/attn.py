"""The attention mixer that stands beside the gated delta rule in a hybrid model (C ABI in ``include/gdr_attn.h``): rotary
positions, softmax attention with its backward, its single-token step over a paged cache, and the write of a prompt into
such a cache.  Checks, streams, workspaces, packed batches and errors as in ``block``.

    rope_forward, rope_backward, rope_frequencies, rope        (autograd), rope_workspace
    attn_forward, attn_backward, attention                     (autograd), attn_workspace
    attn_step, attn_step_workspace                             one token per row over a paged cache
    cache_write, cache_write_workspace                         a prompt's keys and values into it

Served, a sequence's keys and values lie in pages of a pool [num_pages, page_size, Hk, D]; block_table [B, max_pages]
names each row's pages in order:

    q, k = rope_forward(q, k, freqs, cu_seqlens=cu)                     # the prompt
    o, _ = attn_forward(q, k, v, cu_seqlens=cu)
    cache_write(k, v, k_cache, v_cache, block_table, cu_seqlens=cu)
    q, k = rope_forward(q, k, freqs, positions=lengths)                 # then token by token: q, k, v [B, H, D]
    o = attn_step(q, k, v, k_cache, v_cache, block_table, lengths)
    lengths += 1

bf16 tensors whose base and token strides are multiples of 16 bytes run on the tensor cores, others on the CUDA cores, at a fiftieth of the rate
(whatever torch allocates, and slices of it along tokens and heads, are such multiples; a view that begins at an odd element is not).  Values
are taken as finite within a sequence: a NaN or an infinity at a masked place may still reach queries that do not see it, through a
product with a probability of zero.  It reaches no other sequence, and what a cache holds behind a row's end reaches nobody.

Captured into a CUDA graph, a backward pass needs leaves whose earlier eager graphs are gone: autograd adds a leaf's gradient on the
stream that it was first used on while such a graph lives, and that stream is not part of the capture.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._autograd import first_order
from .block import _binding, _done, _gdr, _on, _rows_ok

_c = ctypes
_P, _I, _LL, _SZ, _F = _c.c_void_p, _c.c_int, _c.c_longlong, _c.c_size_t, _c.c_float


class gdr_rope_problem(_c.Structure):
    _fields_ = [("B", _I), ("T", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("R", _I), ("num_seqs", _I), ("cu_seqlens", _P),
                ("dtype", _I), ("interleaved", _I), ("inverse", _I), ("scale", _F), ("ld_q", _LL), ("ld_k", _LL)]


class gdr_attn_problem(_c.Structure):
    _fields_ = [("B", _I), ("Tq", _I), ("Tk", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("num_seqs", _I), ("cu_q", _P),
                ("cu_k", _P), ("dtype", _I), ("causal", _I), ("window", _I), ("scale", _F), ("ld_q", _LL), ("ld_k", _LL),
                ("ld_v", _LL), ("ld_do", _LL)]


class gdr_cache_problem(_c.Structure):
    _fields_ = [("B", _I), ("T", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("num_pages", _I), ("page_size", _I),
                ("max_pages", _I), ("cu_seqlens", _P), ("dtype", _I), ("window", _I), ("scale", _F), ("ld_q", _LL),
                ("ld_k", _LL), ("ld_v", _LL)]


# name: (problem, argument types after it, result type)
SIGNATURES = {
    "gdr_rope_workspace_bytes": (gdr_rope_problem, [], _SZ),
    "gdr_rope": (gdr_rope_problem, [_P] * 7 + [_SZ, _P], _I),
    "gdr_attn_fwd_workspace_bytes": (gdr_attn_problem, [], _SZ),
    "gdr_attn_bwd_workspace_bytes": (gdr_attn_problem, [], _SZ),
    "gdr_attn_fwd": (gdr_attn_problem, [_P] * 6 + [_SZ, _P], _I),
    "gdr_attn_bwd": (gdr_attn_problem, [_P] * 10 + [_SZ, _P], _I),
    "gdr_attn_step_workspace_bytes": (gdr_cache_problem, [], _SZ),
    "gdr_attn_step": (gdr_cache_problem, [_P] * 9 + [_SZ, _P], _I),
    "gdr_cache_write_workspace_bytes": (gdr_cache_problem, [], _SZ),
    "gdr_cache_write": (gdr_cache_problem, [_P] * 7 + [_SZ, _P], _I),
}
ATTN_EXPORTS = sorted(SIGNATURES)


def _clear_workspace(name, p, device):
    nbytes = getattr(_gdr._lib_handle(), name)(_c.byref(p))
    ws = _gdr.alloc_workspace(nbytes, device)
    ws[:256].zero_()  # the status is that of a call; of a problem that needs no workspace it stays clear
    return ws


def _cu(cu):
    return (None, None) if cu is None else (cu.numel() - 1, cu.data_ptr())


# -------------------------------------------------------------------------------- rotary positions
def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=4096, beta_fast=32.0, beta_slow=1.0,
                     device="cuda"):
    """Frequencies of rotary_dim / 2 pairs, base^(-2 i / rotary_dim) radians per position, and the scale that goes with
    them: (freqs float64 [rotary_dim / 2], scale), as rope takes them.

    scaling, for contexts `factor` times as long as the trained one:
      None      as they are
      "linear"  all divided by factor (positions interpolated)
      "ntk"     the base grown so that the slowest pair is factor times as slow and the fastest as it was
      "yarn"    pairs that turn beta_fast times or more over original_length stay, those that turn beta_slow times or less are
                divided by factor, those between are mixed in proportion to their turns; scale 0.1 ln(factor) + 1
                (a model that was tuned with a ramp over the pairs' indices between the two rounded bounds has other frequencies
                between them: hand those to rope as they are)
    """
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim {rotary_dim}: even and above 0")
    if factor < 1.0 or base <= 1.0:
        raise ValueError(f"base {base} and factor {factor}: above 1, and 1 or more")
    half = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    scale = 1.0
    if scaling == "ntk":
        last = half[-1].item()  # base'^-last = base^-last / factor
        base = base * factor ** (1.0 / last) if last else base
    freqs = float(base) ** -half
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "yarn":
        if not beta_fast > beta_slow:
            raise ValueError(f"beta_fast {beta_fast} is not above beta_slow {beta_slow}")
        turns = original_length * freqs / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        freqs = freqs * keep + freqs / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling {scaling!r}: None, 'linear', 'ntk' or 'yarn'")
    return freqs.to(device), scale


def rope_forward(q, k, freqs, positions=None, cu_seqlens=None, interleaved=False, scale=1.0, stream=None, workspace=None):
    """Rotates the first 2 * len(freqs) features of every head of q [B, T, Hq, D] and k [B, T, Hk, D] (or None) by
    position * freqs (float64, radians per position) and multiplies them by scale; the others are passed on.  Pairs are half a rotation apart
    (i, i + R / 2), or neighbours (2 i, 2 i + 1) if interleaved.  positions: int32 [B, T]; None: a token's place in its
    sequence.  Single tokens: q [B, Hq, D], k [B, Hk, D], positions [B].  q and k may be slices of one projection.
    Returns (q, k), rotated."""
    if stream is not None:
        with _on(stream, q):
            return rope_forward(q, k, freqs, positions, cu_seqlens, interleaved, scale, workspace=workspace)
    return _done(_binding().rope(q, k, freqs, positions, cu_seqlens, bool(interleaved), 0, scale, workspace), "gdr_rope")


def rope_backward(dq, dk, freqs, positions=None, cu_seqlens=None, interleaved=False, scale=1.0, stream=None, workspace=None):
    """Gradients of rope_forward from those of its outputs: (dq, dk)."""
    if stream is not None:
        with _on(stream, dq):
            return rope_backward(dq, dk, freqs, positions, cu_seqlens, interleaved, scale, workspace=workspace)
    return _done(_binding().rope(dq, dk, freqs, positions, cu_seqlens, bool(interleaved), 1, scale, workspace), "gdr_rope")


def rope_workspace(q, cu_seqlens=None):
    """A workspace for rope_forward and rope_backward of these tensors, its status word clear."""
    n, at = _cu(cu_seqlens)
    p = gdr_rope_problem(q.shape[0], q.shape[1], q.shape[2], 0, q.shape[3], 2, q.shape[0] if n is None else n, at,
                         _gdr._dtype_code(q.dtype), 0, 0, 1.0)
    return _clear_workspace("gdr_rope_workspace_bytes", p, q.device)


class _RopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, freqs, positions, cu_seqlens, interleaved, scale, workspace):
        ctx.save_for_backward(freqs, positions, cu_seqlens)
        ctx.how = interleaved, scale
        ctx.shapes = q.shape, None if k is None else k.shape
        ctx.like = q.dtype, q.device
        ctx.set_materialize_grads(False)
        return rope_forward(q, k, freqs, positions, cu_seqlens, interleaved, scale, workspace=workspace)

    @staticmethod
    @first_order("rope")
    def backward(ctx, dq, dk):
        freqs, positions, cu = ctx.saved_tensors

        def given(t, shape):
            return torch.zeros(shape, dtype=ctx.like[0], device=ctx.like[1]) if t is None else _rows_ok(t, 2)

        dq = given(dq, ctx.shapes[0])
        dk = given(dk, ctx.shapes[1]) if ctx.shapes[1] is not None else None
        dq, dk = rope_backward(dq, dk, freqs, positions, cu, *ctx.how)
        return dq, dk, None, None, None, None, None, None


def rope(q, k, freqs, positions=None, cu_seqlens=None, interleaved=False, scale=1.0, workspace=None):
    """Autograd entry point of the rotary positions: (q, k) as rope_forward.  freqs and positions have no gradient."""
    return _RopeFunction.apply(q, k, freqs, positions, cu_seqlens, interleaved, scale, workspace)


# --------------------------------------------------------------------------------------- attention
def _scale(scale):
    if scale is not None and not 2.0 ** -126 <= scale < 2.0 ** 128:  # (what rounds to 0 would mean the default)
        raise ValueError(f"scale {scale}: above 0 and in the range of 32 bits, or None for 1 / sqrt(D)")
    return 0.0 if scale is None else scale


def attn_forward(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, window=0, scale=None, stream=None, workspace=None):
    """Softmax attention: q [B, Tq, Hq, D], k and v [B, Tk, Hk, D], Hq a multiple of Hk (query head h reads key head
    h // (Hq // Hk)).  Of n queries and m keys of a sequence, query i sees key j if j <= i + m - n (causal) and
    j > i + m - n - window (window > 0; fewer than 2^31 - 1024 queries and window together, unless it is as wide as the keys).  Packed batches: cu_seqlens of the queries, cu_seqlens_k of the keys where they differ.
    Returns (o [B, Tq, Hq, D], lse [B, Hq, Tq] fp32, the log of the sum of exponentials); a query that sees no key has o = 0 and
    lse = -infinity."""
    if stream is not None:
        with _on(stream, q):
            return attn_forward(q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace=workspace)
    return _done(_binding().attn_forward(q, k, v, cu_seqlens, cu_seqlens_k, bool(causal), window, _scale(scale), workspace),
                 "gdr_attn_fwd")


def attn_backward(q, k, v, o, lse, do, cu_seqlens=None, cu_seqlens_k=None, causal=True, window=0, scale=None, stream=None,
                  workspace=None):
    """Gradients of attn_forward's o from its results o and lse and the gradient do: (dq, dk, dv)."""
    if stream is not None:
        with _on(stream, q):
            return attn_backward(q, k, v, o, lse, do, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace=workspace)
    return _done(_binding().attn_backward(q, k, v, o, lse, do, cu_seqlens, cu_seqlens_k, bool(causal), window, _scale(scale),
                                          workspace), "gdr_attn_bwd")


def attn_workspace(q, k, cu_seqlens=None, cu_seqlens_k=None, backward=False):
    """A workspace for attn_forward (or attn_backward) of these tensors, its status word clear."""
    n, at = _cu(cu_seqlens)
    at_k = at if cu_seqlens_k is None else cu_seqlens_k.data_ptr()
    p = gdr_attn_problem(q.shape[0], q.shape[1], k.shape[1], q.shape[2], k.shape[2], q.shape[3], q.shape[0] if n is None else n, at,
                         at_k, _gdr._dtype_code(q.dtype))
    return _clear_workspace(f"gdr_attn_{'bwd' if backward else 'fwd'}_workspace_bytes", p, q.device)


class _AttnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace):
        o, lse = attn_forward(q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace=workspace)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, cu_seqlens_k)
        ctx.how = causal, window, scale
        return o

    @staticmethod
    @first_order("attention")
    def backward(ctx, do):
        q, k, v, o, lse, cu, cu_k = ctx.saved_tensors
        dq, dk, dv = attn_backward(q, k, v, o, lse, _rows_ok(do, 2), cu, cu_k, *ctx.how)
        return dq, dk, dv, None, None, None, None, None, None


def attention(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal=True, window=0, scale=None, workspace=None):
    """Autograd entry point of attention: o as attn_forward.  workspace: the forward's."""
    return _AttnFunction.apply(q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale, workspace)


# ----------------------------------------------------------------------------------- a paged cache
def attn_step(q, k, v, k_cache, v_cache, block_table, lengths, window=0, scale=None, stream=None, workspace=None):
    """Attention of one token per row: q [B, Hq, D], k and v [B, Hk, D]; k_cache and v_cache [num_pages, page_size, Hk, D];
    block_table int32 [B, max_pages], a row's pages in order; lengths int32 [B], the positions that a row's cache holds.  k and v are
    written at position lengths[b] of their row, and its query attends to positions 0 .. lengths[b] (with a window to the last
    `window` of them).  Returns o [B, Hq, D].  A row whose length is negative or fills its table is skipped and returns zeros;
    one that needs a page outside the pool returns zeros, too (k and v are written if their own page is in the pool).  Rows may read the
    same pages, but no two may write to the same place: rows that fill a batch up have a length of -1.  lengths itself
    is the caller's to advance.  workspace: of attn_step_workspace, for its status."""
    if stream is not None:
        with _on(stream, q):
            return attn_step(q, k, v, k_cache, v_cache, block_table, lengths, window, scale, workspace=workspace)
    return _done(_binding().attn_step(q, k, v, k_cache, v_cache, block_table, lengths, window, _scale(scale), workspace), "gdr_attn_step")


def attn_step_workspace(q, k_cache, block_table):
    """A workspace for attn_step of these tensors, its status word clear."""
    p = gdr_cache_problem(q.shape[0], 1, q.shape[1], k_cache.shape[2], q.shape[2], k_cache.shape[0], k_cache.shape[1],
                          block_table.shape[1], None, _gdr._dtype_code(q.dtype))
    return _clear_workspace("gdr_attn_step_workspace_bytes", p, q.device)


def cache_write(k, v, k_cache, v_cache, block_table, starts=None, cu_seqlens=None, stream=None, workspace=None):
    """Writes k and v [B, T, Hk, D] (packed: [1, T, Hk, D]) into their sequences' pages from position starts[n] (int32 [B];
    None: 0) on; cache and block_table as attn_step, a row of the table per sequence.  Tokens whose position or page does not exist
    are left out; no two may go to the same place."""
    if stream is not None:
        with _on(stream, k):
            return cache_write(k, v, k_cache, v_cache, block_table, starts, cu_seqlens, workspace=workspace)
    return _done(_binding().cache_write(k, v, k_cache, v_cache, block_table, starts, cu_seqlens, workspace), "gdr_cache_write")


def cache_write_workspace(k, cu_seqlens=None):
    """A workspace for cache_write of these tensors, its status word clear."""
    n, at = _cu(cu_seqlens)
    p = gdr_cache_problem(k.shape[0] if n is None else n, k.shape[1], 0, k.shape[2], k.shape[3], 0, 1, 0, at,
                          _gdr._dtype_code(k.dtype))
    return _clear_workspace("gdr_cache_write_workspace_bytes", p, k.device)
