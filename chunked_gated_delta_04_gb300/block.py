"""The operators around the gated delta rule (C ABI in ``include/gdr_block.h``): the short causal
convolution, the selective state space scan, the block norms and the single-token step.

As in the package's main module the functions with a C name marshal arguments and return the
status; the others check shapes, types and strides, allocate outputs and workspace and raise
(``ValueError`` for what they find themselves, ``GDRError`` for a status).  Everything runs on the
current stream, or on ``stream`` if one is given: outputs and workspace are then allocated on that
stream, and the caller orders the inputs before it.

    conv_forward, conv_backward, conv_step, causal_conv        (autograd)
    ssm_forward, ssm_backward, ssm_step, selective_scan        (autograd)
    norm_forward, norm_backward, block_norm                    (autograd)
    step                                                       the gated delta rule, one token
"""
from __future__ import annotations

import ctypes
import sys

import torch

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


_gdr = sys.modules[__package__]  # the package itself, which imports this module


def _lib():
    return _gdr._LIB or _gdr._lib_handle()


def _raise(status, where):
    raise _gdr.GDRError(status, where)


_CODE = {torch.float32: 0, torch.bfloat16: 1}
_F32 = torch.float32
_empty = torch.empty


def _on(stream):
    """The context in which a call on a stream of its own allocates and launches."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


# The current stream's handle.  torch.cuda.current_stream() builds an object for it (2.9 us on the
# GPU's host, against 2.7 us for a whole launch through the library); the raw query takes 0.1 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _p(t):
    return None if t is None else t.data_ptr()


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _is(t, shape, dtype=_F32):
    """Whether t is a contiguous CUDA tensor of a shape and type (None passes)."""
    return t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda)


def _act(name, t, shape, dtype):
    """An activation of the call: on the GPU, of the call's type and shape."""
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _full(name, t, shape, dtype=torch.float32):
    """A contiguous tensor of a given shape and type, or None."""
    if not _is(t, shape, dtype):
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _ld(name, t, inner):
    """Token stride of a [B, T, ...inner] activation (0: contiguous); its rows must be contiguous and
    evenly spaced over the batch."""
    if t.is_contiguous():
        return 0
    shape, st = t.shape, t.stride()
    width = 1
    for k in range(len(shape) - 1, len(shape) - 1 - inner, -1):
        _need(shape[k] == 1 or st[k] == width, f"{name}: rows must be contiguous (strides {st})")
        width *= shape[k]
    lead = [k for k in range(len(shape) - inner) if shape[k] != 1]
    if not lead:
        return 0
    ld = st[lead[-1]]
    for a, b in zip(lead, lead[1:]):
        _need(st[a] == st[b] * shape[b], f"{name}: the batch must be evenly strided (strides {st})")
    _need(ld >= width, f"{name}: token stride {ld} below the row width {width}")
    return ld


def _seqs(cu_seqlens, B):
    if cu_seqlens is None:
        return B
    if B == 1 and cu_seqlens.dtype is torch.int32 and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous():
        n = cu_seqlens.numel()
        if n >= 2 and cu_seqlens.is_cuda:
            return n - 1
    _need(cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda and cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2
          and cu_seqlens.is_contiguous(), "cu_seqlens: expected a contiguous CUDA int32 vector of at least 2 entries")
    _need(B == 1, "cu_seqlens needs a batch of 1 (the packed tokens)")
    return cu_seqlens.numel() - 1


def _slots(slots, B):
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (B,) or not slots.is_cuda
                              or not slots.is_contiguous()):
        raise ValueError(f"slots: expected a contiguous CUDA int32 vector of {B} entries")


def _workspace(nbytes, device):
    # torch's allocator returns 512-byte aligned blocks, which covers the 256-byte requirement
    return _empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _type(x):
    code = _CODE.get(x.dtype)
    if code is None:
        raise ValueError(f"dtype {x.dtype}: float32 or bfloat16")
    return code


_LAYOUT = {"KV": 0, "VK": 1}
_I32 = torch.int32


def _slots_ok(slots, n, B):
    if slots is None:
        return n >= B
    return slots.dtype is _I32 and slots.shape == (B,) and slots.is_contiguous() and slots.is_cuda


def _step_state(state, slots, B):
    _slots(slots, B)
    if slots is None and state.shape[0] < B:
        raise ValueError(f"state: {state.shape[0]} states for {B} rows")


# ---------------------------------------------------------------------------------- convolution
_SILU = {"silu": 1, "none": 0, None: 0}


def _silu(activation):
    if activation not in _SILU:
        raise ValueError(f"activation {activation!r}: 'silu' or 'none'")
    return _SILU[activation]


def _conv_problem(x, weight, bias, cu_seqlens, activation, state, name, dy=None):
    if x.dim() != 3:
        raise ValueError(f"x: expected [B, T, C], got {tuple(x.shape)}")
    B, T, C = x.shape
    W = weight.shape[-1]
    _act("x", x, (B, T, C), x.dtype)
    _full("weight", weight, (C, W))
    _full("bias", bias, (C,))
    N = _seqs(cu_seqlens, B)
    _full(name, state, (N, W - 1, C), x.dtype)
    ld_dy = 0
    if dy is not None:
        _act("dy", dy, (B, T, C), x.dtype)
        ld_dy = _ld("dy", dy, 1)
    return gdr_conv_problem(B, T, C, W, N, _p(cu_seqlens), _type(x), _silu(activation), _ld("x", x, 1), ld_dy, 0)


def conv_forward(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu", output_final_state=False,
                 stream=None):
    """Short causal depthwise convolution: x [B, T, C] (may be a slice of a wider tensor), weight
    [C, W] and bias [C] fp32, initial_state [num_seqs, W - 1, C] (oldest row first).  Returns
    (y, final state or None)."""
    if stream is not None:
        with _on(stream):
            return conv_forward(x, weight, bias, initial_state, cu_seqlens, activation, output_final_state)
    p = _conv_problem(x, weight, bias, cu_seqlens, activation, initial_state, "initial_state")
    lib = _lib()
    y = _empty(x.shape, dtype=x.dtype, device=x.device)
    last = (_empty(p.num_seqs, p.W - 1, p.C, dtype=x.dtype, device=x.device) if output_final_state else None)
    ws = _workspace(256 if cu_seqlens is not None else 0, x.device)
    st = lib.gdr_conv_fwd(p, _p(x), _p(weight), _p(bias), _p(initial_state), _p(y), _p(last), _p(ws),
                          256 if ws is not None else 0, _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_conv_fwd")
    return y, last


def conv_backward(x, weight, bias, dy, initial_state=None, dfinal_state=None, cu_seqlens=None, activation="silu",
                  stream=None):
    """Gradients of conv_forward: (dx, dweight, dbias or None, dinitial_state or None)."""
    if stream is not None:
        with _on(stream):
            return conv_backward(x, weight, bias, dy, initial_state, dfinal_state, cu_seqlens, activation)
    p = _conv_problem(x, weight, bias, cu_seqlens, activation, initial_state, "initial_state", dy)
    _full("dfinal_state", dfinal_state, (p.num_seqs, p.W - 1, p.C), x.dtype)
    lib = _lib()
    dx = _empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    dstate = torch.empty_like(initial_state) if initial_state is not None else None
    n = lib.gdr_conv_bwd_workspace_bytes(p)
    ws = _workspace(n, x.device)
    st = lib.gdr_conv_bwd(p, _p(x), _p(weight), _p(bias), _p(initial_state), _p(dy), _p(dfinal_state), _p(dx),
                          _p(dw), _p(db), _p(dstate), _p(ws), n, _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_conv_bwd")
    return dx, dw, db, dstate


def conv_step(x, state, weight, bias=None, slots=None, activation="silu", stream=None):
    """One token per row: x [B, C]; state, a pool [num_slots, W - 1, C], is updated in place at each
    row's slot (int32 [B]; None: row i at slot i).  Returns y [B, C]; a row whose slot is outside the
    pool is skipped and returns zeros."""
    if stream is not None:
        with _on(stream):
            return conv_step(x, state, weight, bias, slots, activation)
    dtype = x.dtype
    B, C = x.shape
    n, W, c = state.shape
    W += 1
    ld = 0
    # the usual call passes here; anything else is named by the checks
    if not (c == C and state.dtype is dtype and weight.dtype is _F32 and weight.shape == (C, W) and x.is_contiguous()
            and state.is_contiguous() and weight.is_contiguous() and x.is_cuda and state.is_cuda and weight.is_cuda
            and dtype in _CODE and (bias is None or _is(bias, (C,))) and _slots_ok(slots, n, B) and activation in _SILU):
        _act("x", x, (B, C), dtype)
        _full("weight", weight, (C, W))
        _full("bias", bias, (C,))
        _full("state", state, (n, W - 1, C), dtype)
        _step_state(state, slots, B)
        _type(x)
        _silu(activation)
        ld = _ld("x", x, 1)
    p = gdr_conv_problem(B, 1, C, W, B, None, _CODE[dtype], _SILU[activation], ld, 0, n)
    y = _empty((B, C), dtype=dtype, device=x.device) if ld else torch.empty_like(x)
    st = _lib().gdr_conv_step(p, x.data_ptr(), weight.data_ptr(), _p(bias), state.data_ptr(), _p(slots), y.data_ptr(),
                              _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_conv_step")
    return y


class _ConvFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation):
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return conv_forward(x, weight, bias, initial_state, cu_seqlens, activation, output_final_state=True)

    @staticmethod
    def backward(ctx, dy, dlast):
        x, weight, bias, state, cu = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _rows_ok(dy, 1)
        dx, dw, db, dstate = conv_backward(x, weight, bias, dy, state, None if dlast is None else dlast.contiguous(), cu,
                                           ctx.activation)
        return dx, dw, db, dstate, None, None


def _rows_ok(t, inner):
    """t if a call can take its strides, else a contiguous copy."""
    try:
        _ld("", t, inner)
        return t
    except ValueError:
        return t.contiguous()


def causal_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation="silu"):
    """Autograd entry point of the short causal convolution: (y, final state).  weight and bias may
    be of any float type (they are used in fp32)."""
    return _ConvFunction.apply(x, weight.float(), None if bias is None else bias.float(), initial_state, cu_seqlens,
                               activation)


# ------------------------------------------------------------------------------- selective scan
def _ssm_problem(x, dt, A, Bm, Cm, Dskip, dt_bias, cu_seqlens, dt_softplus, dy=None):
    if x.dim() != 3 or Bm.dim() != 4:
        raise ValueError(f"expected x [B, T, D] and Bm, Cm [B, T, G, N], got {tuple(x.shape)} and {tuple(Bm.shape)}")
    B, T, D = x.shape
    G, N = Bm.shape[2], Bm.shape[3]
    _act("x", x, (B, T, D), x.dtype)
    _act("dt", dt, (B, T, D), x.dtype)
    _act("Bm", Bm, (B, T, G, N), x.dtype)
    _act("Cm", Cm, (B, T, G, N), x.dtype)
    _full("A", A, (D, N))
    _full("D", Dskip, (D,))
    _full("dt_bias", dt_bias, (D,))
    ld_dy = 0
    if dy is not None:
        _act("dy", dy, (B, T, D), x.dtype)
        ld_dy = _ld("dy", dy, 1)
    return gdr_ssm_problem(B, T, D, N, G, _seqs(cu_seqlens, B), _p(cu_seqlens), _type(x), int(bool(dt_softplus)),
                           _ld("x", x, 1), _ld("dt", dt, 1), _ld("Bm", Bm, 2), _ld("Cm", Cm, 2), ld_dy, 0)


def ssm_forward(x, dt, A, Bm, Cm, D=None, dt_bias=None, S0=None, cu_seqlens=None, dt_softplus=True,
                output_final_state=True, save=True, stream=None):
    """Selective state space scan: x, dt [B, T, D], A [D, N] fp32, Bm, Cm [B, T, G, N], D and dt_bias
    [D] fp32, S0 [num_seqs, D, N] fp32.  Returns (y, S_T or None, h_saved or None); save keeps the
    states that ssm_backward needs."""
    if stream is not None:
        with _on(stream):
            return ssm_forward(x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus, output_final_state, save)
    p = _ssm_problem(x, dt, A, Bm, Cm, D, dt_bias, cu_seqlens, dt_softplus)
    _full("S0", S0, (p.num_seqs, p.D, p.N))
    lib = _lib()
    y = _empty(x.shape, dtype=x.dtype, device=x.device)
    S_T = _empty((p.num_seqs, p.D, p.N), dtype=torch.float32, device=x.device) if output_final_state else None
    saved = None
    if save:
        saved = _empty(lib.gdr_ssm_saved_bytes(p) // 4, dtype=torch.float32, device=x.device)
    n = lib.gdr_ssm_fwd_workspace_bytes(p)
    ws = _workspace(n, x.device)
    st = lib.gdr_ssm_fwd(p, _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(dt_bias), _p(S0), _p(y), _p(S_T),
                         _p(saved), _p(ws), n, _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_ssm_fwd")
    return y, S_T, saved


def ssm_backward(x, dt, A, Bm, Cm, h_saved, dy, D=None, dt_bias=None, dS_T=None, cu_seqlens=None, dt_softplus=True,
                 want_dS0=True, stream=None):
    """Gradients of ssm_forward: (dx, ddt, dA, dBm, dCm, dD or None, ddt_bias or None, dS0 or None)."""
    if stream is not None:
        with _on(stream):
            return ssm_backward(x, dt, A, Bm, Cm, h_saved, dy, D, dt_bias, dS_T, cu_seqlens, dt_softplus, want_dS0)
    p = _ssm_problem(x, dt, A, Bm, Cm, D, dt_bias, cu_seqlens, dt_softplus, dy)
    _full("dS_T", dS_T, (p.num_seqs, p.D, p.N))
    lib = _lib()
    need = lib.gdr_ssm_saved_bytes(p) // 4
    if h_saved is None or h_saved.dtype != _F32 or not h_saved.is_contiguous() or h_saved.numel() < need:
        raise ValueError(f"h_saved: expected the {need} floats that ssm_forward kept (save=True)")
    f32 = torch.float32
    dx, ddt = (_empty(x.shape, dtype=x.dtype, device=x.device) for _ in range(2))
    dB, dC = (_empty(Bm.shape, dtype=x.dtype, device=x.device) for _ in range(2))
    dA = torch.empty_like(A)
    dD = torch.empty_like(D) if D is not None else None
    dbias = torch.empty_like(dt_bias) if dt_bias is not None else None
    dS0 = _empty((p.num_seqs, p.D, p.N), dtype=f32, device=x.device) if want_dS0 else None
    n = lib.gdr_ssm_bwd_workspace_bytes(p)
    ws = _workspace(n, x.device)
    st = lib.gdr_ssm_bwd(p, _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(dt_bias), _p(h_saved), _p(dy),
                         _p(dS_T), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC), _p(dD), _p(dbias), _p(dS0), _p(ws), n,
                         _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_ssm_bwd")
    return dx, ddt, dA, dB, dC, dD, dbias, dS0


def ssm_step(x, dt, A, Bm, Cm, state, D=None, dt_bias=None, slots=None, dt_softplus=True, stream=None):
    """One token per row: x, dt [B, D], Bm, Cm [B, G, N]; state, a pool [num_slots, D, N] fp32, is
    updated in place at each row's slot (see conv_step).  Returns y [B, D]."""
    if stream is not None:
        with _on(stream):
            return ssm_step(x, dt, A, Bm, Cm, state, D, dt_bias, slots, dt_softplus)
    dtype = x.dtype
    B, d = x.shape
    _, G, N = Bm.shape
    n = state.shape[0]
    lds = (0, 0, 0, 0)
    if not (dt.dtype is dtype and Bm.dtype is dtype and Cm.dtype is dtype and dt.shape == (B, d) and Bm.shape == (B, G, N)
            and Cm.shape == (B, G, N) and x.is_contiguous() and dt.is_contiguous() and Bm.is_contiguous()
            and Cm.is_contiguous() and x.is_cuda and dt.is_cuda and Bm.is_cuda and Cm.is_cuda and dtype in _CODE
            and _is(A, (d, N)) and _is(state, (n, d, N)) and (D is None or _is(D, (d,)))
            and (dt_bias is None or _is(dt_bias, (d,))) and _slots_ok(slots, n, B)):
        _act("x", x, (B, d), dtype)
        _act("dt", dt, (B, d), dtype)
        _act("Bm", Bm, (B, G, N), dtype)
        _act("Cm", Cm, (B, G, N), dtype)
        _full("A", A, (d, N))
        _full("D", D, (d,))
        _full("dt_bias", dt_bias, (d,))
        _full("state", state, (n, d, N))
        _step_state(state, slots, B)
        _type(x)
        lds = (_ld("x", x, 1), _ld("dt", dt, 1), _ld("Bm", Bm, 2), _ld("Cm", Cm, 2))
    p = gdr_ssm_problem(B, 1, d, N, G, B, None, _CODE[dtype], 1 if dt_softplus else 0, *lds, 0, n)
    y = _empty((B, d), dtype=dtype, device=x.device)
    st = _lib().gdr_ssm_step(p, x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _p(D), _p(dt_bias),
                             state.data_ptr(), _p(slots), y.data_ptr(), _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_ssm_step")
    return y


class _SSMFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus):
        y, S_T, saved = ssm_forward(x, dt, A, Bm, Cm, D, dt_bias, S0, cu_seqlens, dt_softplus)
        ctx.save_for_backward(x, dt, A, Bm, Cm, D, dt_bias, saved, cu_seqlens)
        ctx.dt_softplus, ctx.has_S0 = dt_softplus, S0 is not None
        ctx.set_materialize_grads(False)
        return y, S_T

    @staticmethod
    def backward(ctx, dy, dS_T):
        x, dt, A, Bm, Cm, D, dt_bias, saved, cu = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _rows_ok(dy, 1)
        grads = ssm_backward(x, dt, A, Bm, Cm, saved, dy, D, dt_bias, None if dS_T is None else dS_T.contiguous(), cu,
                             ctx.dt_softplus, want_dS0=ctx.has_S0)
        return (*grads, None, None)


def selective_scan(x, dt, A, Bm, Cm, D=None, dt_bias=None, initial_state=None, cu_seqlens=None, dt_softplus=True):
    """Autograd entry point of the selective scan: (y, final state).  A, D and dt_bias may be of any
    float type (they are used in fp32)."""
    def f(t):
        return None if t is None else t.float()

    return _SSMFunction.apply(x, dt, f(A), Bm, Cm, f(D), f(dt_bias), initial_state, cu_seqlens, dt_softplus)


# ---------------------------------------------------------------------------------- block norms
def _norm_rows(x, gate):
    """(tokens, heads, ld_x, ld_gate): rows are the last dimension; a tensor of heads may be a slice
    of a wider one (its tokens strided, its heads side by side)."""
    D = x.shape[-1]
    if (x.is_contiguous()) and (gate is None or gate.is_contiguous()):
        return x.numel() // D if D else 0, 1, 0, 0
    err = None
    for inner in (1, 2) if x.dim() > 2 else (1,):
        heads = 1 if inner == 1 else x.shape[-2]
        try:
            ld = [0 if t is None else _ld(n, t, inner) for n, t in (("x", x), ("gate", gate))]
            return x.numel() // (D * heads), heads, ld[0], ld[1]
        except ValueError as e:
            err = e
    raise err


def _norm_problem(x, post_weight, gate, scale, pre_weight, stream_dtype, eps):
    D = x.shape[-1]
    _act("x", x, x.shape, x.dtype)
    if gate is not None:
        _act("gate", gate, x.shape, x.dtype)
    _full("post_weight", post_weight, (D,))
    _full("scale", scale, (D,))
    _full("pre_weight", pre_weight, (D,))
    tokens, heads, ld_x, ld_gate = _norm_rows(x, gate)
    if stream_dtype not in _CODE:
        raise ValueError(f"residual dtype {stream_dtype}: float32 or bfloat16")
    return gdr_norm_problem(tokens, heads, D, _type(x), _CODE[stream_dtype], eps, ld_x, ld_gate)


def norm_forward(x, post_weight=None, gate=None, scale=None, residual=None, pre_weight=None, eps=1e-6, stream=None):
    """u = x [rstd(x) post_weight] [silu(gate)] [scale]; r = [residual +] u; y = r rstd(r) pre_weight.
    Rows are the last dimension.  Returns (r, y): r in the residual's dtype (fp32 or x's), or in x's
    without one; r is None for a plain norm in front of a block (pre_weight alone), y is None without
    pre_weight."""
    if stream is not None:
        with _on(stream):
            return norm_forward(x, post_weight, gate, scale, residual, pre_weight, eps)
    dtype, shape = x.dtype, x.shape
    res_dtype = dtype if residual is None else residual.dtype
    D = shape[-1]
    if (x.is_contiguous() and x.is_cuda and dtype in _CODE and res_dtype in _CODE and D > 0
            and (gate is None or _is(gate, shape, dtype)) and (residual is None or _is(residual, shape, res_dtype))
            and (post_weight is None or _is(post_weight, (D,))) and (scale is None or _is(scale, (D,)))
            and (pre_weight is None or _is(pre_weight, (D,)))):
        p = gdr_norm_problem(x.numel() // D, 1, D, _CODE[dtype], _CODE[res_dtype], eps, 0, 0)
    else:
        p = _norm_problem(x, post_weight, gate, scale, pre_weight, res_dtype, eps)
        _full("residual", residual, shape, res_dtype)
    r = y = None
    if residual is not None:
        r = torch.empty_like(residual)
    elif pre_weight is None:
        r = _empty(shape, dtype=dtype, device=x.device)
    if pre_weight is not None:
        y = _empty(shape, dtype=dtype, device=x.device)
    st = _lib().gdr_norm_fwd(p, x.data_ptr(), _p(post_weight), _p(gate), _p(scale), _p(residual), _p(pre_weight), _p(r), _p(y),
                             _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_norm_fwd")
    return r, y


def norm_backward(x, post_weight=None, gate=None, scale=None, r=None, pre_weight=None, dr=None, dy=None, eps=1e-6,
                  stream=None):
    """Gradients of norm_forward from dr and dy (either may be None): (dx, dgate, dresidual, dpost_weight,
    dscale, dpre_weight), None where the forward had no such tensor.  r: the forward's r where it had a
    residual, else None."""
    if stream is not None:
        with _on(stream):
            return norm_backward(x, post_weight, gate, scale, r, pre_weight, dr, dy, eps)
    has_residual = r is not None
    res_dtype = r.dtype if has_residual else x.dtype
    p = _norm_problem(x, post_weight, gate, scale, pre_weight, res_dtype, eps)
    _full("r", r, x.shape, res_dtype)
    _full("dr", dr, x.shape, res_dtype)
    _full("dy", dy, x.shape, x.dtype)
    if not has_residual and pre_weight is not None:
        _need(x.is_contiguous(), "x: a plain norm's backward needs a contiguous x")
    lib = _lib()

    def new(like, dtype=None):
        return None if like is None else _empty(like.shape, dtype=dtype or like.dtype, device=x.device)

    dx, dgate = new(x), new(gate)
    dres = new(x, res_dtype) if has_residual else None
    dpost, dscale, dpre = new(post_weight), new(scale), new(pre_weight)
    n = lib.gdr_norm_bwd_workspace_bytes(p)
    ws = _workspace(n, x.device)
    rr = r if has_residual else (x if pre_weight is not None else None)
    st = lib.gdr_norm_bwd(p, _p(x), _p(post_weight), _p(gate), _p(scale), _p(rr), _p(pre_weight),
                          int(has_residual), _p(dr), _p(dy), _p(dx), _p(dgate), _p(dres), _p(dpost), _p(dscale), _p(dpre),
                          _p(ws), n, _raw_stream(x.get_device()))
    if st:
        _raise(st, "gdr_norm_bwd")
    return dx, dgate, dres, dpost, dscale, dpre


class _NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, post_weight, gate, scale, residual, pre_weight, eps):
        r, y = norm_forward(x, post_weight, gate, scale, residual, pre_weight, eps)
        ctx.save_for_backward(x, post_weight, gate, scale, r if residual is not None else None, pre_weight)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return r, y

    @staticmethod
    def backward(ctx, dr, dy):
        x, post_weight, gate, scale, r, pre_weight = ctx.saved_tensors
        if pre_weight is not None and dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
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
def step(q, k, v, g, beta, state, layout="KV", scale=None, slots=None, prologue=0, stream=None):
    """The gated delta rule for one token per row: q, k [B, Hk, DK], v [B, Hv, DV], g [B, Hv] fp32,
    beta [B, Hv]; state, a pool [num_slots, Hv, DK, DV] ("KV") or [num_slots, Hv, DV, DK] ("VK") fp32,
    is updated in place at each row's slot (see conv_step).  prologue: GDR_PROLOGUE_* bits, as in
    forward (the mapped q, k and beta stay in fp32 here).  Returns o [B, Hv, DV]."""
    if stream is not None:
        with _on(stream):
            return step(q, k, v, g, beta, state, layout, scale, slots, prologue)
    dtype = q.dtype
    B, Hk, DK = q.shape
    Hv, DV = v.shape[1:]
    n = state.shape[0]
    if not (_is(q, (B, Hk, DK), dtype) and _is(k, (B, Hk, DK), dtype) and _is(v, (B, Hv, DV), dtype) and _is(g, (B, Hv))
            and _is(beta, (B, Hv), dtype) and layout in _LAYOUT and dtype in _CODE and _slots_ok(slots, n, B)
            and _is(state, (n, Hv, DK, DV) if layout == "KV" else (n, Hv, DV, DK))):
        if layout not in _LAYOUT:
            raise ValueError(f"layout {layout!r}: 'KV' or 'VK'")
        _type(q)
        _full("q", q, (B, Hk, DK), dtype)
        _full("k", k, (B, Hk, DK), dtype)
        _full("v", v, (B, Hv, DV), dtype)
        _full("g", g, (B, Hv))
        _full("beta", beta, (B, Hv), dtype)
        _full("state", state, (n, Hv, DK, DV) if layout == "KV" else (n, Hv, DV, DK))
        _step_state(state, slots, B)
    p = _gdr.gdr_problem(B, 1, Hk, Hv, DK, DV, B, None, _CODE[dtype], _LAYOUT[layout], 0.0 if scale is None else scale, 0,
                         prologue, 0, 1, 1)
    o = torch.empty_like(v)
    st = _lib().gdr_step(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(), n,
                         _p(slots), o.data_ptr(), _raw_stream(q.get_device()))
    if st:
        _raise(st, "gdr_step")
    return o
