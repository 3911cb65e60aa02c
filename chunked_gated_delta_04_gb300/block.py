"""The operators around the gated delta rule (C ABI in ``include/gdr_block.h``): the short causal
convolution, the selective state space scan, the block norms and the single-token step.

The functions here check shapes, types and strides, allocate outputs and workspace and make the call
(in ``csrc/gdr_binding.cpp``), and raise: ``ValueError`` for what they find themselves, ``GDRError`` for
a status.  A call's tensors lie on one device, whichever is current, and the call runs there.  Everything runs on
its current stream, or on ``stream`` if one is given: outputs and workspace are then allocated on that stream, and the
caller orders the inputs before it and keeps them until it is done.

Packed batches (``cu_seqlens``): what cu_seqlens holds is checked on the device.  A malformed one (not 0 .. T in
non-decreasing steps) computes nothing, the outputs are then uninitialised, and the workspace's status says so.  To be
able to ask, hand a workspace in and ask after the call:

    ws = conv_workspace(x, weight, cu_seqlens)
    y, last = conv_forward(x, weight, cu_seqlens=cu_seqlens, workspace=ws)
    status, flags = gdr_workspace_status(ws)   # synchronises; GDR_ERR_INVALID_ARG

    conv_forward, conv_backward, conv_step, causal_conv        (autograd), conv_workspace
    ssm_forward, ssm_backward, ssm_step, selective_scan        (autograd), ssm_workspace
    norm_forward, norm_backward, block_norm                    (autograd)
    step                                                       the gated delta rule, one token
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import sys

import torch

from ._autograd import first_order, link

_c = ctypes
_P, _I, _LL, _SZ, _F = _c.c_void_p, _c.c_int, _c.c_longlong, _c.c_size_t, _c.c_float


class gdr_conv_problem(_c.Structure):
    _fields_ = [("B", _I), ("T", _I), ("C", _I), ("W", _I), ("num_seqs", _I), ("cu_seqlens", _P), ("dtype", _I),
                ("silu", _I), ("ld_x", _LL), ("ld_dy", _LL), ("num_slots", _I)]


class gdr_ssm_problem(_c.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("N", _I), ("G", _I), ("num_seqs", _I), ("cu_seqlens", _P),
                ("dtype", _I), ("dt_softplus", _I), ("ld_x", _LL), ("ld_dt", _LL), ("ld_b", _LL), ("ld_c", _LL),
                ("ld_dy", _LL), ("num_slots", _I)]


class gdr_norm_problem(_c.Structure):
    _fields_ = [("tokens", _LL), ("heads", _I), ("D", _I), ("dtype", _I), ("res_dtype", _I), ("eps", _F),
                ("ld_x", _LL), ("ld_gate", _LL)]


# name: (argument types after the problem, result type); the sizes come from here too
_SIGNATURES = {
    "gdr_conv_fwd_workspace_bytes": (gdr_conv_problem, [], _SZ),
    "gdr_conv_bwd_workspace_bytes": (gdr_conv_problem, [], _SZ),
    "gdr_conv_fwd": (gdr_conv_problem, [_P] * 7 + [_SZ, _P], _I),
    "gdr_conv_bwd": (gdr_conv_problem, [_P] * 11 + [_SZ, _P], _I),
    "gdr_conv_step": (gdr_conv_problem, [_P] * 7, _I),
    "gdr_ssm_saved_bytes": (gdr_ssm_problem, [], _SZ),
    "gdr_ssm_fwd_workspace_bytes": (gdr_ssm_problem, [], _SZ),
    "gdr_ssm_bwd_workspace_bytes": (gdr_ssm_problem, [], _SZ),
    "gdr_ssm_fwd": (gdr_ssm_problem, [_P] * 12 + [_SZ, _P], _I),
    "gdr_ssm_bwd": (gdr_ssm_problem, [_P] * 19 + [_SZ, _P], _I),
    "gdr_ssm_step": (gdr_ssm_problem, [_P] * 11, _I),
    "gdr_norm_fwd": (gdr_norm_problem, [_P] * 9, _I),
    "gdr_norm_bwd_workspace_bytes": (gdr_norm_problem, [], _SZ),
    "gdr_norm_bwd": (gdr_norm_problem, [_P] * 6 + [_I] + [_P] * 9 + [_SZ, _P], _I),
}
BLOCK_EXPORTS = sorted(_SIGNATURES) + ["gdr_step"]


def declare(lib, gdr_problem) -> None:
    """C signatures of this module's entry points, on a library the main module opens."""
    for name, (problem, args, result) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = [_c.POINTER(problem)] + args
        fn.restype = result
    lib.gdr_step.argtypes = [_c.POINTER(gdr_problem)] + [_P] * 6 + [_I] + [_P] * 3
    lib.gdr_step.restype = _I
    for name, (problem, args, result) in _attn().SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = [_c.POINTER(problem)] + args
        fn.restype = result


def _attn():
    from . import attn  # which imports this module

    return attn


_gdr = sys.modules[__package__]  # the package itself, which imports this module
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "gdr_binding.so")
_module = _bound = None


def _binding():
    """The torch binding, bound to the library that the package has open."""
    global _module, _bound
    lib = _gdr._LIB or _gdr._lib_handle()
    if _bound is not lib:
        if _module is None:
            if not os.path.exists(BINDING_PATH):
                raise ImportError(f"gdr_binding.so not built ({BINDING_PATH}); run `python -m {__package__}.build`")
            loader = importlib.machinery.ExtensionFileLoader("gdr_binding", BINDING_PATH)
            spec = importlib.util.spec_from_loader("gdr_binding", loader)
            _module = importlib.util.module_from_spec(spec)
            loader.exec_module(_module)
        _module.bind({n: _c.cast(getattr(lib, n), _c.c_void_p).value for n in BLOCK_EXPORTS + _attn().ATTN_EXPORTS})
        _bound = lib
    return _module


def _done(result, where):
    """A call's outputs, or GDRError for the status in their place."""
    if type(result) is int:
        raise _gdr.GDRError(result, where)
    return result


def _on(stream, x):
    """The context in which a call with tensor x on a stream of its own allocates and launches; a handle (int) is one
    of x's device."""
    device = x.device if isinstance(x, torch.Tensor) and x.is_cuda else None  # else the call says what x is
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    elif device is not None and stream.device != device:
        raise ValueError(f"stream: of {stream.device}, the call's first tensor on {device}")
    return torch.cuda.stream(stream)


def _ld(name, t, inner):
    """Token stride of a [B, T, ...inner] activation (0: contiguous); its rows must be contiguous and
    evenly spaced over the batch."""
    ld = _binding().stride(t, inner)
    if ld < 0:
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced over the batch (shape {tuple(t.shape)}, "
                         f"strides {t.stride()})")
    return ld


# ---------------------------------------------------------------------------------- convolution
_SILU = {"silu": 1, "none": 0, None: 0}


def _silu(activation):
    if activation not in _SILU:
        raise ValueError(f"activation {activation!r}: 'silu' or 'none'")
    return _SILU[activation]


def conv_forward(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu", output_final_state=False,
                 stream=None, workspace=None):
    """Short causal depthwise convolution: x [B, T, C] (may be a slice of a wider tensor), weight
    [C, W] and bias [C] fp32, initial_state [num_seqs, W - 1, C] (oldest row first).  Returns
    (y, final state or None).  workspace: of conv_workspace, for its status."""
    if stream is not None:
        with _on(stream, x):
            return conv_forward(x, weight, bias, initial_state, cu_seqlens, activation, output_final_state,
                                workspace=workspace)
    return _done(_binding().conv_forward(x, weight, bias, initial_state, cu_seqlens, _silu(activation), output_final_state,
                                         workspace), "gdr_conv_fwd")


def conv_backward(x, weight, bias, dy, initial_state=None, dfinal_state=None, cu_seqlens=None, activation="silu",
                  stream=None, workspace=None):
    """Gradients of conv_forward: (dx, dweight, dbias or None, dinitial_state or None)."""
    if stream is not None:
        with _on(stream, x):
            return conv_backward(x, weight, bias, dy, initial_state, dfinal_state, cu_seqlens, activation,
                                 workspace=workspace)
    return _done(_binding().conv_backward(x, weight, bias, dy, initial_state, dfinal_state, cu_seqlens, _silu(activation),
                                          workspace), "gdr_conv_bwd")


def conv_workspace(x, weight, cu_seqlens=None, backward=False):
    """A workspace for conv_forward (or conv_backward) of these tensors, its status word clear."""
    B, T, C = x.shape
    cu = cu_seqlens
    p = gdr_conv_problem(B, T, C, weight.shape[-1], B if cu is None else cu.numel() - 1, None if cu is None else cu.data_ptr(),
                         _gdr._dtype_code(x.dtype))
    return _workspace("conv", p, backward, x.device)


def _workspace(op, p, backward, device):
    nbytes = getattr(_gdr._lib_handle(), f"gdr_{op}_{'bwd' if backward else 'fwd'}_workspace_bytes")(_c.byref(p))
    ws = _gdr.alloc_workspace(nbytes, device)
    ws[:256].zero_()  # the status is a packed call's; of another it stays clear
    return ws


def conv_step(x, state, weight, bias=None, slots=None, activation="silu", stream=None):
    """One token per row: x [B, C]; state, a pool [num_slots, W - 1, C], is updated in place at each
    row's slot (int32 [B]; None: row i at slot i).  Returns y [B, C]; a row whose slot is outside the
    pool is skipped and returns zeros."""
    if stream is not None:
        with _on(stream, x):
            return conv_step(x, state, weight, bias, slots, activation)
    return _done(_binding().conv_step(x, state, weight, bias, slots, _silu(activation)), "gdr_conv_step")


class _ConvFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation, workspace):
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return conv_forward(x, weight, bias, initial_state, cu_seqlens, activation, output_final_state=True, workspace=workspace)

    @staticmethod
    @first_order("causal_conv")
    def backward(ctx, dy, dlast):
        x, weight, bias, state, cu = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _rows_ok(dy, 1)
        dx, dw, db, dstate = conv_backward(x, weight, bias, dy, state, None if dlast is None else dlast.contiguous(), cu,
                                           ctx.activation)
        return dx, dw, db, dstate, None, None, None


def _rows_ok(t, inner):
    """t if a call can take its strides, else a contiguous copy."""
    return t if _binding().stride(t, inner) >= 0 else t.contiguous()


def causal_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu", workspace=None):
    """Autograd entry point of the short causal convolution: (y, final state).  weight and bias may
    be of any float type (they are used in fp32).  workspace: the forward's, as conv_forward."""
    return _ConvFunction.apply(x, weight.float(), None if bias is None else bias.float(), initial_state, cu_seqlens,
                               activation, workspace)


# ------------------------------------------------------------------------------- selective scan
def ssm_forward(x, dt, A, Bm, Cm, D=None, dt_bias=None, S0=None, cu_seqlens=None, dt_softplus=True,
                output_final_state=True, save=True, stream=None, workspace=None):
    """Selective state space scan: x, dt [B, T, D], A [D, N] fp32, Bm, Cm [B, T, G, N], D and dt_bias
    [D] fp32, S0 [num_seqs, D, N] fp32.  Returns (y, S_T or None, h_saved or None); save keeps the
    states that ssm_backward needs.  workspace: of ssm_workspace, for its status."""
    if stream is not None:
        with _on(stream, x):
            return ssm_forward(x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus, output_final_state, save,
                               workspace=workspace)
    return _done(_binding().ssm_forward(x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, bool(dt_softplus), output_final_state,
                                        save, workspace), "gdr_ssm_fwd")


def ssm_backward(x, dt, A, Bm, Cm, h_saved, dy, D=None, dt_bias=None, dS_T=None, cu_seqlens=None, dt_softplus=True,
                 want_dS0=True, stream=None, workspace=None):
    """Gradients of ssm_forward: (dx, ddt, dA, dBm, dCm, dD or None, ddt_bias or None, dS0 or None)."""
    if stream is not None:
        with _on(stream, x):
            return ssm_backward(x, dt, A, Bm, Cm, h_saved, dy, D, dt_bias, dS_T, cu_seqlens, dt_softplus, want_dS0,
                                workspace=workspace)
    return _done(_binding().ssm_backward(x, dt, A, Bm, Cm, h_saved, dy, D, dt_bias, dS_T, cu_seqlens, bool(dt_softplus),
                                         want_dS0, workspace), "gdr_ssm_bwd")


def ssm_workspace(x, Bm, cu_seqlens=None, backward=False):
    """A workspace for ssm_forward (or ssm_backward) of these tensors, its status word clear."""
    B, T, D = x.shape
    cu = cu_seqlens
    p = gdr_ssm_problem(B, T, D, Bm.shape[-1], Bm.shape[-2], B if cu is None else cu.numel() - 1,
                        None if cu is None else cu.data_ptr(), _gdr._dtype_code(x.dtype))
    return _workspace("ssm", p, backward, x.device)


def ssm_step(x, dt, A, Bm, Cm, state, D=None, dt_bias=None, slots=None, dt_softplus=True, stream=None):
    """One token per row: x, dt [B, D], Bm, Cm [B, G, N]; state, a pool [num_slots, D, N] fp32, is
    updated in place at each row's slot (see conv_step).  Returns y [B, D]."""
    if stream is not None:
        with _on(stream, x):
            return ssm_step(x, dt, A, Bm, Cm, state, D, dt_bias, slots, dt_softplus)
    return _done(_binding().ssm_step(x, dt, A, Bm, Cm, state, D, dt_bias, slots, bool(dt_softplus)), "gdr_ssm_step")


class _SSMFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus, S0_link, workspace):
        y, S_T, saved = ssm_forward(x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus, workspace=workspace)
        ctx.save_for_backward(x, dt, A, Bm, Cm, D, dt_bias, saved, cu_seqlens, S0_link)
        ctx.dt_softplus, ctx.has_S0 = dt_softplus, S0 is not None
        ctx.set_materialize_grads(False)
        return y, S_T

    @staticmethod
    @first_order("selective_scan")
    def backward(ctx, dy, dS_T):
        x, dt, A, Bm, Cm, D, dt_bias, saved, cu, _ = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _rows_ok(dy, 1)
        grads = ssm_backward(x, dt, A, Bm, Cm, saved, dy, D, dt_bias, None if dS_T is None else dS_T.contiguous(), cu,
                             ctx.dt_softplus, want_dS0=ctx.has_S0)
        return (*grads, None, None, None, None)


def selective_scan(x, dt, A, Bm, Cm, D=None, dt_bias=None, initial_state=None, cu_seqlens=None, dt_softplus=True,
                   workspace=None):
    """Autograd entry point of the selective scan: (y, final state).  A, D and dt_bias may be of any
    float type (they are used in fp32).  workspace: the forward's, as ssm_forward."""
    def f(t):
        return None if t is None else t.float()

    return _SSMFunction.apply(x, dt, f(A), Bm, Cm, f(D), f(dt_bias), initial_state, cu_seqlens, dt_softplus,
                              link(initial_state), workspace)


# ---------------------------------------------------------------------------------- block norms
def norm_forward(x, post_weight=None, gate=None, scale=None, residual=None, pre_weight=None, eps=1e-6, stream=None):
    """u = x [rstd(x) post_weight] [silu(gate)] [scale]; r = [residual +] u; y = r rstd(r) pre_weight.
    Rows are the last dimension.  Returns (r, y): r in the residual's dtype (fp32 or x's), or in x's
    without one; r is None for a plain norm in front of a block (pre_weight alone), y is None without
    pre_weight."""
    if stream is not None:
        with _on(stream, x):
            return norm_forward(x, post_weight, gate, scale, residual, pre_weight, eps)
    return _done(_binding().norm_forward(x, post_weight, gate, scale, residual, pre_weight, eps), "gdr_norm_fwd")


def norm_backward(x, post_weight=None, gate=None, scale=None, r=None, pre_weight=None, dr=None, dy=None, eps=1e-6,
                  stream=None):
    """Gradients of norm_forward from dr and dy, the gradients of the outputs that it had (of two, either may be
    None): (dx, dgate, dresidual, dpost_weight, dscale, dpre_weight), None where the forward had no such tensor.
    r: the forward's r where it had a residual, else None."""
    if stream is not None:
        with _on(stream, x):
            return norm_backward(x, post_weight, gate, scale, r, pre_weight, dr, dy, eps)
    if dy is None and dr is not None and pre_weight is not None and r is not None:  # the library wants it with pre_weight
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    return _done(_binding().norm_backward(x, post_weight, gate, scale, r, pre_weight, dr, dy, eps), "gdr_norm_bwd")


class _NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, post_weight, gate, scale, residual, pre_weight, eps):
        r, y = norm_forward(x, post_weight, gate, scale, residual, pre_weight, eps)
        ctx.save_for_backward(x, post_weight, gate, scale, r if residual is not None else None, pre_weight)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return r, y

    @staticmethod
    @first_order("block_norm")
    def backward(ctx, dr, dy):
        x, post_weight, gate, scale, r, pre_weight = ctx.saved_tensors
        if pre_weight is not None and dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        if pre_weight is not None and r is None:  # a plain norm's backward takes x as the r it was applied to
            x = x.contiguous()
        if pre_weight is None and dr is None:
            dr = torch.zeros(x.shape, dtype=x.dtype if r is None else r.dtype, device=x.device)
        dx, dgate, dres, dpost, dscale, dpre = norm_backward(
            x, post_weight, gate, scale, r, pre_weight, None if dr is None else dr.contiguous(),
            None if dy is None else dy.contiguous(), ctx.eps)
        return dx, dpost, dgate, dscale, dres, dpre, None


def block_norm(x, post_weight=None, gate=None, scale=None, residual=None, pre_weight=None, eps=1e-6):
    """Autograd entry point of the block norms: (r, y) as norm_forward.  Weights and scale may be of
    any float type (they are used in fp32)."""
    def f(t):
        return None if t is None else t.float()

    return _NormFunction.apply(x, f(post_weight), gate, f(scale), residual, f(pre_weight), eps)


# ----------------------------------------------------------------- the delta rule, one token each
_LAYOUT = {"KV": 0, "VK": 1}


def step(q, k, v, g, beta, state, layout="KV", scale=None, slots=None, prologue=0, stream=None):
    """The gated delta rule for one token per row: q, k [B, Hk, DK], v [B, Hv, DV], g [B, Hv] fp32,
    beta [B, Hv]; state, a pool [num_slots, Hv, DK, DV] ("KV") or [num_slots, Hv, DV, DK] ("VK") fp32,
    is updated in place at each row's slot (see conv_step).  scale: None (or not above 0) is 1 / sqrt(DK).  prologue:
    GDR_PROLOGUE_* bits, as in forward (the mapped q, k and beta stay in fp32 here).  Returns o [B, Hv, DV]."""
    if stream is not None:
        with _on(stream, q):
            return step(q, k, v, g, beta, state, layout, scale, slots, prologue)
    if layout not in _LAYOUT:
        raise ValueError(f"layout {layout!r}: 'KV' or 'VK'")
    return _done(_binding().step(q, k, v, g, beta, state, _LAYOUT[layout], 0.0 if scale is None else scale, slots, prologue),
                 "gdr_step")
