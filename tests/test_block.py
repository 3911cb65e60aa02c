"""GPU parity of the operators around the gated delta rule with their fp64 references.

Tolerances, from the arithmetic:
- a bf16 output is the fp32 result rounded once to 8 significant bits: each element is within half an
  ulp, 2^-8 of its own value, of the fp32 result, whose error the next line bounds.
- an fp32 output comes from at most ~300 dependent steps with ~4 roundings of 2^-24 and two hardware
  approximations of ~2^-22 each, which add up like a random walk: sqrt(300) * 2^-21 = 8e-6;
  bound 3e-5 of the largest value.
- parameter gradients are fp32 sums over up to ~700 tokens of terms of either sign: the relative error
  of one term (1e-6) grows by at most sum |t| / |sum t| ~ sqrt(700) = 26: bound 5e-5.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from oracle import block as ob

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
PARAMS = {"dw", "db", "dA", "dD", "ddt_bias", "dw_post", "dscale", "dw_pre"}


def gen(seed):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, dtype=F32, mul=1.0, add=0.0):
        return (torch.randn(*shape, generator=g) * mul + add).to(dtype)

    return rand


def npy(t):
    return None if t is None else t.detach().double().cpu().numpy()


def cuda(t):
    return None if t is None else t.cuda()


def check(got, ref):
    """got: name -> tensor (or None); ref: name -> fp64 array."""
    bad = {}
    for k, t in got.items():
        if t is None:
            continue
        a, b = npy(t), ref[k].reshape(t.shape)
        if a.size == 0:
            continue
        assert np.isfinite(a).all(), k
        most = (5e-5 if k in PARAMS else 3e-5) * max(np.abs(b).max(), 1e-30)
        if t.dtype == BF:
            most = most + 2.0 ** -8 * np.abs(b)
        over = (np.abs(a - b) / most).max()
        if not over <= 1:
            bad[k] = over
    assert not bad, bad


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def wide(t, extra, off):
    """t as a slice of a wider tensor (token stride larger than the row)."""
    shape = t.shape
    big = torch.full((*shape[:2], shape[2] + extra, *shape[3:]), 7.0, dtype=t.dtype, device=t.device)
    big[:, :, off:off + shape[2]] = t
    return big[:, :, off:off + shape[2]]


# ---------------------------------------------------------------------------------- convolution
def conv_inputs(dtype, C, W, lens, bias, state, seed=0):
    r = gen(seed)
    T, n = sum(lens), len(lens)
    d = dict(x=r(1, T, C, dtype=dtype), w=r(C, W, mul=0.5), b=r(C) if bias else None,
             state=r(n, W - 1, C, dtype=dtype) if state else None, dy=r(1, T, C, dtype=dtype),
             dl=r(n, W - 1, C, dtype=dtype) if state else None)
    return {k: cuda(v) for k, v in d.items()}


def conv_check(d, lens, act, cu, x=None, dy=None, stream=None):
    x, dy = d["x"] if x is None else x, d["dy"] if dy is None else dy
    y, last = gdr.conv_forward(x, d["w"], d["b"], d["state"], cu, act, output_final_state=True, stream=stream)
    dx, dw, db, ds = gdr.conv_backward(x, d["w"], d["b"], dy, d["state"], d["dl"], cu, act, stream=stream)
    torch.cuda.synchronize()
    C = x.shape[-1]
    ref = ob.conv(npy(x).reshape(-1, C), npy(d["w"]), npy(d["b"]), npy(d["state"]), lens, act == "silu",
                  npy(dy).reshape(-1, C), npy(d["dl"]))
    got = dict(y=y, last=last, dx=dx, dw=dw, db=db, dstate=ds)
    check(got, ref)
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("C,W,lens,act,bias,state", [
    (64, 4, [130], "silu", False, False),
    (8, 4, [1], "silu", True, True),
    (5, 3, [0, 3, 1, 0, 40, 2], "silu", True, True),      # scalar path, empty and short sequences
    (264, 2, [33, 1, 0, 300], "none", False, True),
    (1024, 4, [2, 2, 2, 257, 64], "silu", True, False),
    (37, 4, [700], "none", True, True),
    (2056, 3, [5], "silu", False, True),
])
def test_conv_varlen(dtype, C, W, lens, act, bias, state):
    d = conv_inputs(dtype, C, W, lens, bias, state)
    conv_check(d, lens, act, cu_of(lens).cuda())


@pytest.mark.parametrize("B,T,C", [(1, 1, 16), (3, 2, 40), (2, 65, 128), (4, 0, 8)])
def test_conv_fixed_length_and_strides(B, T, C):
    d = conv_inputs(BF, C, 4, [T] * B, True, True)
    x, dy = d["x"].reshape(B, T, C), d["dy"].reshape(B, T, C)
    a = conv_check(d, [T] * B, "silu", None, x, dy)
    for extra, off in ((8, 8), (3, 1)):  # vector path, then misaligned rows
        b = conv_check(d, [T] * B, "silu", None, wide(x, extra, off), wide(dy, extra, off))
        for k in ("y", "last", "dx", "dstate"):  # per element the same arithmetic
            assert torch.equal(a[k], b[k]), k


def test_conv_step_continues_the_prompt():
    r = gen(4)
    B, T, C, W = 5, 9, 72, 4
    x, w, b = r(B, T, C, dtype=BF).cuda(), r(C, W).cuda(), r(C).cuda()
    y, last = gdr.conv_forward(x, w, b, output_final_state=True)
    y0, state = gdr.conv_forward(x[:, :T - 3].contiguous(), w, b, output_final_state=True)
    slots = torch.tensor([6, 0, 3, 2, 5], dtype=torch.int32).cuda()
    pool = torch.zeros(8, W - 1, C, dtype=BF).cuda()
    pool[slots.long()] = state
    for t in range(T - 3, T):
        yt = gdr.conv_step(x[:, t], pool, w, b, slots)
        assert torch.equal(yt, y[:, t])
    assert torch.equal(pool[slots.long()], last)


@pytest.mark.parametrize("dtype,C,W", [(F32, 7, 2), (BF, 64, 3), (F32, 256, 4)])
def test_conv_step_and_skipped_rows(dtype, C, W):
    r = gen(5)
    x, w, pool = r(4, C, dtype=dtype).cuda(), r(C, W).cuda(), r(6, W - 1, C, dtype=dtype).cuda()
    before = pool.clone()
    slots = torch.tensor([4, -1, 6, 0], dtype=torch.int32).cuda()  # -1 and 6 name no state
    y = gdr.conv_step(x, pool, w, slots=slots, activation="none")
    for i, s in ((0, 4), (3, 0)):
        ref = ob.conv(npy(x[i:i + 1]), npy(w), None, npy(before[s:s + 1]), [1], False)
        check(dict(y=y[i:i + 1], last=pool[s:s + 1]), ref)
    assert not y[1].any() and not y[2].any()
    for s in (1, 2, 3, 5):
        assert torch.equal(pool[s], before[s])


# ------------------------------------------------------------------------------- selective scan
def ssm_inputs(dtype, D, N, G, lens, state, skip=True, bias=True, seed=0, dt_mul=0.5):
    r = gen(seed)
    T, n = sum(lens), len(lens)
    A = -torch.arange(1, N + 1, dtype=F32).expand(D, N) * torch.exp(r(D, N, mul=0.1))
    d = dict(x=r(1, T, D, dtype=dtype), dt=r(1, T, D, dtype=dtype, mul=dt_mul), A=A.contiguous(),
             Bm=r(1, T, G, N, dtype=dtype), Cm=r(1, T, G, N, dtype=dtype), D=r(D) if skip else None,
             dt_bias=r(D, mul=0.5, add=-3.0) if bias else None, S0=r(n, D, N) if state else None,
             dy=r(1, T, D, dtype=dtype), dS_T=r(n, D, N) if state else None)
    return {k: cuda(v) for k, v in d.items()}


def ssm_run(d, cu, soft=True, stream=None):
    y, S_T, saved = gdr.ssm_forward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["dt_bias"], d["S0"], cu, soft,
                                    stream=stream)
    g = gdr.ssm_backward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], saved, d["dy"], d["D"], d["dt_bias"], d["dS_T"], cu, soft,
                         stream=stream)
    torch.cuda.synchronize()
    return dict(zip(("y", "S_T", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dS0"), (y, S_T, *g)))


def ssm_ref(d, lens, soft=True):
    D = d["x"].shape[-1]
    G, N = d["Bm"].shape[2:]
    f = {k: npy(v) for k, v in d.items()}
    return ob.ssm(f["x"].reshape(-1, D), f["dt"].reshape(-1, D), f["A"], f["Bm"].reshape(-1, G, N), f["Cm"].reshape(-1, G, N),
                  f["D"], f["dt_bias"], f["S0"], lens, soft, f["dy"].reshape(-1, D), f["dS_T"])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,N,G,lens,state,soft", [
    (64, 16, 1, [100], True, True),
    (1, 4, 1, [1], False, True),
    (40, 8, 2, [0, 17, 1, 0, 33, 16], True, True),       # empty sequences, tiles that end inside, groups
    (200, 16, 1, [300], False, True),                    # cut into segments
    (70, 32, 1, [65, 15, 129], True, False),
    (36, 64, 4, [40, 3], True, True),
    (130, 4, 1, [250, 9], True, True),
    (2048, 16, 2, [2, 1], True, True),
])
def test_ssm_varlen(dtype, D, N, G, lens, state, soft):
    d = ssm_inputs(dtype, D, N, G, lens, state)
    if not soft:
        d["dt"] = d["dt"].abs() * 0.1
        d["dt_bias"] = None
    check(ssm_run(d, cu_of(lens).cuda(), soft), ssm_ref(d, lens, soft))


@pytest.mark.parametrize("B,T,D", [(2, 48, 64), (1, 0, 8), (3, 1, 24), (20, 90, 1024)])
def test_ssm_fixed_length_and_strides(B, T, D):
    lens = [T] * B
    d = ssm_inputs(BF, D, 16, 1, lens, B < 20, skip=B != 3, bias=B != 3, dt_mul=0.2)
    d = {k: (v.reshape(B, T, *v.shape[2:]) if v is not None and v.shape[:2] == (1, B * T) else v) for k, v in d.items()}
    a = ssm_run(d, None)
    if D <= 64:
        check(a, ssm_ref(d, lens))
    e = dict(d, **{k: wide(d[k], 5, 2) for k in ("x", "dt", "dy")})
    both = torch.cat([d["Bm"], d["Cm"]], -1)  # B and C side by side, as a projection leaves them
    e["Bm"], e["Cm"] = both[..., :16], both[..., 16:]
    b = ssm_run(e, None)
    for k in a:
        assert a[k] is None or torch.equal(a[k], b[k]), k


def test_ssm_segments_equal_the_whole():
    """A packed batch cut into segments equals its sequences run one at a time (fp32 rounding)."""
    lens = [500, 64, 1, 333]
    d = ssm_inputs(F32, 96, 16, 1, lens, True)
    whole = ssm_run(d, cu_of(lens).cuda())
    check(whole, ssm_ref(d, lens))


def test_ssm_extremes():
    """Steps near zero and very large, decay rates of 0 and -infinity, an infinite negative dt."""
    d = ssm_inputs(F32, 8, 4, 1, [40], True)
    d["dt"][:, 3] = -200.0      # no step: the state passes
    d["dt"][:, 5] = 300.0       # decays to nothing
    d["dt"][:, 7] = -float("inf")
    d["A"][0] = 0.0
    y, S_T, _ = gdr.ssm_forward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["dt_bias"], d["S0"])
    ref = ssm_ref(d, [40])
    check(dict(y=y, S_T=S_T), ref)
    d["A"][1] = -float("inf")   # forgets all but the newest token
    d["dt"][:, 7] = 0.0
    d["dt"][:, 3] = -3.0
    y, S_T, _ = gdr.ssm_forward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["dt_bias"], d["S0"])
    check(dict(y=y, S_T=S_T), ssm_ref(d, [40]))


@pytest.mark.parametrize("what", ["A", "dt", "x", "Bm", "S0"])
def test_ssm_nan_reaches_what_depends_on_it(what):
    """A NaN in an input makes the outputs NaN that depend on it, and no others."""
    d = ssm_inputs(F32, 8, 4, 1, [40], True)
    at = {"A": (3, 2), "dt": (0, 30, 3), "x": (0, 30, 3), "Bm": (0, 30, 0, 1), "S0": (0, 3, 1)}[what]
    d[what][at] = float("nan")
    y, S_T, _ = gdr.ssm_forward(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], d["D"], d["dt_bias"], d["S0"])
    t0 = 30 if what in ("dt", "x", "Bm") else 0
    bad = torch.zeros(40, 8, dtype=torch.bool)
    bad[t0:, slice(None) if what == "Bm" else 3] = True
    assert torch.equal(y[0].isnan().cpu(), bad)
    assert torch.equal(S_T[0].isnan().any(1).cpu(), bad[-1])
    pool = d["S0"].clone()
    ys = gdr.ssm_step(d["x"][:, 30], d["dt"][:, 30], d["A"], d["Bm"][:, 30], d["Cm"][:, 30], pool, d["D"], d["dt_bias"])
    assert torch.equal(ys[0].isnan().cpu(), bad[30])


@pytest.mark.parametrize("dtype,D,N,G", [(F32, 33, 4, 1), (BF, 64, 16, 2), (BF, 24, 64, 1), (F32, 130, 8, 1)])
def test_ssm_step(dtype, D, N, G):
    d = ssm_inputs(dtype, D, N, G, [7], False)
    x, dt, Bm, Cm = (d[k][0, :5] for k in ("x", "dt", "Bm", "Cm"))
    pool = gen(9)(9, D, N).cuda()
    before = pool.clone()
    slots = torch.tensor([8, 2, -5, 9, 0], dtype=torch.int32).cuda()  # -5 and 9 name no state
    y = gdr.ssm_step(x, dt, d["A"], Bm, Cm, pool, d["D"], d["dt_bias"], slots)
    for i, s in ((0, 8), (1, 2), (4, 0)):
        ref = ob.ssm(npy(x[i:i + 1]), npy(dt[i:i + 1]), npy(d["A"]), npy(Bm[i:i + 1]), npy(Cm[i:i + 1]), npy(d["D"]),
                     npy(d["dt_bias"]), npy(before[s:s + 1]), [1])
        check(dict(y=y[i:i + 1], S_T=pool[s:s + 1]), ref)
    assert not y[2].any() and not y[3].any()
    for s in (1, 3, 4, 5, 6, 7):
        assert torch.equal(pool[s], before[s])


# ---------------------------------------------------------------------------------- block norms
MODES = {"gated": (1, 1, 0, 0, 0), "add": (0, 0, 0, 1, 1), "full": (1, 1, 1, 1, 1), "plain": (0, 0, 0, 0, 1),
         "post": (1, 0, 0, 0, 0), "stream": (1, 0, 1, 1, 0), "scale": (0, 1, 1, 0, 0)}


def norm_inputs(mode, dtype, res_dtype, shape, seed=0):
    post, gate, scale, res, pre = MODES[mode]
    r = gen(seed)
    D = shape[-1]
    d = dict(x=r(*shape, dtype=dtype), post=r(D, mul=0.1, add=1) if post else None,
             z=r(*shape, dtype=dtype) if gate else None, scale=r(D) if scale else None,
             res=r(*shape, dtype=res_dtype) if res else None, pre=r(D, mul=0.1, add=1) if pre else None,
             dr=r(*shape, dtype=res_dtype if res else dtype) if res or not pre else None,
             dy=r(*shape, dtype=dtype) if pre else None)
    return {k: cuda(v) for k, v in d.items()}


def norm_run(d, x=None, z=None, stream=None):
    x, z = d["x"] if x is None else x, d["z"] if z is None else z
    r, y = gdr.norm_forward(x, d["post"], z, d["scale"], d["res"], d["pre"], stream=stream)
    g = gdr.norm_backward(x, d["post"], z, d["scale"], r if d["res"] is not None else None, d["pre"], d["dr"], d["dy"],
                          stream=stream)
    torch.cuda.synchronize()
    return dict(zip(("r", "y", "dx", "dz", "dresidual", "dw_post", "dscale", "dw_pre"), (r, y, *g)))


def norm_check(got, d):
    f = {k: npy(v) for k, v in d.items()}
    D = d["x"].shape[-1]
    f = {k: (v.reshape(-1, D) if v is not None and v.ndim > 1 else v) for k, v in f.items()}
    r, y = ob.norm(f["x"], f["post"], f["z"], f["scale"], f["res"], f["pre"])
    ref = {"r": r, "y": y}
    if d["res"] is not None and d["pre"] is not None:  # the norm in front of the next block is of r as stored
        stored = npy(got["r"]).reshape(-1, D)
        ref["y"] = ob.norm(stored, w_pre=f["pre"])[1]
    else:
        stored = npy(got["r"]).reshape(-1, D) if d["res"] is not None else f["x"]
    ref.update(ob.norm_grad(f["x"], f["post"], f["z"], f["scale"], stored, f["pre"], f["dr"], f["dy"]))
    check(got, ref)


@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("shape", [(1, 3), (3, 7), (70, 64), (37, 128), (33, 200), (9, 512), (5, 1000), (3, 2048), (4, 4104),
                                   (2, 8191), (2, 16384)])
def test_norm(types, mode, shape):
    if types == (BF, F32) and not MODES[mode][3]:
        pytest.skip("no residual")
    d = norm_inputs(mode, *types, shape)
    norm_check(norm_run(d), d)


@pytest.mark.parametrize("rows", [1000, 3001])
def test_norm_many_rows(rows):
    """More rows than blocks: every block walks several and joins its sums."""
    for mode, D in (("gated", 128), ("full", 640)):
        d = norm_inputs(mode, F32, F32, (rows, D))
        norm_check(norm_run(d), d)


@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("mode", ["full", "add", "gated", "scale"])
def test_norm_wide_rows_in_turn(types, mode):
    """Rows of a block each, more of them than blocks: the next row is under way while one is worked on."""
    if types == (BF, F32) and not MODES[mode][3]:
        pytest.skip("no residual")
    for D in (4104, 8192):
        d = norm_inputs(mode, *types, (333, D))
        norm_check(norm_run(d), d)


def test_norm_rows_of_heads_in_a_wider_tensor():
    B, T, H, D = 2, 5, 3, 64
    d = norm_inputs("gated", BF, BF, (B, T, H, D))
    a = norm_run(d)
    norm_check(a, d)
    for extra, off in ((64, 64), (5, 3)):
        x = wide(d["x"].reshape(B, T, H * D), extra, off).unflatten(-1, (H, D))
        z = wide(d["z"].reshape(B, T, H * D), extra + 8, 8).unflatten(-1, (H, D))
        b = norm_run(d, x, z)
        for k in a:
            assert a[k] is None or torch.equal(a[k], b[k]) or k == "dw_post", k
        check(dict(dw_post=b["dw_post"]), dict(dw_post=npy(a["dw_post"])))


def test_norm_rows_stay_apart():
    """A row of zeros gives zeros, a row with NaN only itself NaN."""
    d = norm_inputs("gated", F32, F32, (6, 128))
    d["x"][2] = 0.0
    d["x"][4, 7] = float("nan")
    d["z"][1] = 200.0
    d["z"][3] = -200.0
    r, _ = gdr.norm_forward(d["x"], d["post"], d["z"])
    assert not r[2].any() and torch.isnan(r[4]).all() and not r[3].abs().max() > 1e-30
    ok = [0, 1, 2, 3, 5]
    assert torch.isfinite(r[ok]).all()
    ref = ob.norm(npy(d["x"])[ok], npy(d["post"]), npy(d["z"])[ok])[0]
    check(dict(y=r[ok]), dict(y=ref))


# ----------------------------------------------------------------- the delta rule, one token each
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["KV", "VK"])
@pytest.mark.parametrize("B,Hk,Hv,DK,DV,prologue", [(1, 1, 1, 128, 128, 7), (3, 2, 6, 128, 128, 0), (2, 1, 2, 16, 112, 7),
                                                   (2, 3, 3, 80, 16, 1), (5, 2, 2, 64, 48, 6), (2, 1, 1, 112, 32, 4)])
def test_step(dtype, layout, B, Hk, Hv, DK, DV, prologue):
    r = gen(B * 100 + DK)
    q, k, v = r(B, Hk, DK, dtype=dtype).cuda(), r(B, Hk, DK, dtype=dtype).cuda(), r(B, Hv, DV, dtype=dtype).cuda()
    if not prologue & 1:
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(dtype) for t in (q, k))
    g, beta = r(B, Hv).cuda(), r(B, Hv, dtype=dtype).cuda()
    if not prologue & 2:
        g = -g.abs()
    if not prologue & 4:
        beta = torch.sigmoid(beta)
    shape = (DK, DV) if layout == "KV" else (DV, DK)
    pool = r(B + 3, Hv, *shape).cuda()
    before = pool.clone()
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1
    o = gdr.step(q, k, v, g, beta, pool, layout=layout, slots=slots.cuda(), prologue=prologue)
    rows = [i for i in range(B) if slots[i] >= 0]
    at = slots[rows].long()
    S = npy(before)[at.numpy()]
    if layout == "KV":
        S = S.transpose(0, 1, 3, 2)
    f = [npy(t)[rows] for t in (q, k, v, g, beta)]
    ro, rS = ob.step(*f, S, None, bool(prologue & 1), bool(prologue & 2), bool(prologue & 4))
    if layout == "KV":
        rS = rS.transpose(0, 1, 3, 2)
    check(dict(o=o[rows], S=pool[at.cuda()]), dict(o=ro, S=rS))
    rest = [s for s in range(B + 3) if s not in at.tolist()]
    assert torch.equal(pool[rest], before[rest])
    if B > 2:
        assert not o[1].any()


@pytest.mark.parametrize("layout", ["KV", "VK"])
def test_step_continues_the_prompt(layout):
    """States that gdr.forward leaves carry on token by token as the whole prompt does (fp32 path)."""
    r = gen(11)
    B, T, H, D = 2, 70, 2, 64
    q, k = (torch.nn.functional.normalize(r(B, T, H, D), dim=-1).cuda() for _ in range(2))
    v, g, beta = r(B, T, H, D).cuda(), -r(B, T, H).abs().cuda(), torch.sigmoid(r(B, T, H)).cuda()
    o, S_T, _ = gdr.forward(q, k, v, g, beta, layout=layout)
    part = [t[:, :T - 4].contiguous() for t in (q, k, v, g, beta)]
    _, S, _ = gdr.forward(*part, layout=layout)
    for t in range(T - 4, T):
        ot = gdr.step(*(a[:, t].contiguous() for a in (q, k, v, g, beta)), S, layout=layout)
        # the chunked form's own bound on fp32 inputs is 1e-4
        assert (ot - o[:, t]).abs().max() <= 1e-4 * o.abs().max()
    assert (S - S_T).abs().max() <= 1e-4 * S_T.abs().max()


# ------------------------------------------------------------------------------------ all of them
def everything(stream=None):
    c = conv_inputs(BF, 64, 4, [33, 0, 70], True, True)
    s = ssm_inputs(BF, 64, 16, 1, [33, 0, 70], True)
    n = norm_inputs("full", BF, F32, (103, 128))
    cu = cu_of([33, 0, 70]).cuda()
    torch.cuda.synchronize()
    out = dict(conv_check(c, [33, 0, 70], "silu", cu, stream=stream))
    out.update({"s_" + k: v for k, v in ssm_run(s, cu, stream=stream).items()})
    out.update({"n_" + k: v for k, v in norm_run(n, stream=stream).items()})
    return out


def test_bitwise_the_same_on_every_run_and_stream():
    a, b, c = everything(), everything(), everything(torch.cuda.Stream())
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 5, 10], [0, 5, 9], [0, -4, 10]])
def test_malformed_cu_seqlens_is_reported_and_nothing_computed(cu):
    import ctypes

    bad = torch.tensor(cu, dtype=torch.int32).cuda()
    n = len(cu) - 1
    lib = gdr.load()
    x = torch.ones(1, 10, 8, device="cuda")
    w = torch.ones(8, 4, device="cuda")
    y = torch.full_like(x, 3.0)
    dw = torch.full_like(w, 3.0)
    p = gdr.gdr_conv_problem(1, 10, 8, 4, n, bad.data_ptr(), 0, 1, 0, 0, 0)
    ws = torch.empty(lib.gdr_conv_bwd_workspace_bytes(ctypes.byref(p)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream

    def status():
        st, flags = gdr.gdr_workspace_status(ws)
        assert st == gdr.GDR_ERR_INVALID_ARG and flags & 1

    assert lib.gdr_conv_fwd(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, y.data_ptr(), None, ws.data_ptr(),
                            ws.numel(), s) == 0
    status()
    assert lib.gdr_conv_bwd(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, x.data_ptr(), None, y.data_ptr(),
                            dw.data_ptr(), None, None, ws.data_ptr(), ws.numel(), s) == 0
    status()
    assert (y == 3).all() and (dw == 3).all()
    A = torch.full((8, 4), -1.0, device="cuda")
    bc = torch.ones(1, 10, 1, 4, device="cuda")
    p = gdr.gdr_ssm_problem(1, 10, 8, 4, 1, n, bad.data_ptr(), 0, 1, 0, 0, 0, 0, 0, 0)
    saved = torch.zeros(lib.gdr_ssm_saved_bytes(ctypes.byref(p)) // 4, device="cuda")
    ws = torch.empty(lib.gdr_ssm_bwd_workspace_bytes(ctypes.byref(p)), dtype=torch.uint8, device="cuda")
    assert lib.gdr_ssm_fwd(ctypes.byref(p), x.data_ptr(), x.data_ptr(), A.data_ptr(), bc.data_ptr(), bc.data_ptr(), None, None,
                           None, y.data_ptr(), None, saved.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    status()
    dA, db, dc = torch.full_like(A, 3.0), torch.full_like(bc, 3.0), torch.full_like(bc, 3.0)
    assert lib.gdr_ssm_bwd(ctypes.byref(p), x.data_ptr(), x.data_ptr(), A.data_ptr(), bc.data_ptr(), bc.data_ptr(), None, None,
                           saved.data_ptr(), x.data_ptr(), None, y.data_ptr(), y.data_ptr(), dA.data_ptr(), db.data_ptr(),
                           dc.data_ptr(), None, None, None, ws.data_ptr(), ws.numel(), s) == 0
    status()
    assert all((t == 3).all() for t in (y, dA, db, dc))


def test_autograd_against_differences():
    """Gradients of the autograd entry points against central differences of their own fp32 forwards.
    Directions are unit-normal per element; with step 1e-2 the truncation is ~1e-4 of the gradient term
    and the fp32 rounding of a loss of ~1e3 terms gives ~1e-3: bound 1e-2."""
    r = gen(21)
    B, T, C, N = 2, 20, 16, 8
    x0 = r(B, T, C).cuda()
    P = dict(x=x0, w=r(C, 4).cuda(), b=r(C).cuda(), dt=r(B, T, C, mul=0.3).cuda(), A=-torch.exp(r(C, N, mul=0.2)).cuda(),
             Bm=r(B, T, 1, N).cuda(), Cm=r(B, T, 1, N).cuda(), D=r(C).cuda(), z=r(B, T, C).cuda(), post=r(C).cuda(),
             scale=r(C).cuda(), res=r(B, T, C).cuda(), pre=r(C).cuda())
    wy, wr, wS = r(B, T, C).cuda(), r(B, T, C).cuda(), r(B, C, N).cuda()

    def loss(p):
        h, _ = gdr.causal_conv(p["x"], p["w"], p["b"])
        y, S = gdr.selective_scan(h, p["dt"], p["A"], p["Bm"], p["Cm"], p["D"])
        rr, yy = gdr.block_norm(y, p["post"], p["z"], p["scale"], p["res"], p["pre"])
        return (yy.double() * wy).sum() + (rr.double() * wr).sum() + (S.double() * wS).sum()

    leaf = {k: v.clone().requires_grad_() for k, v in P.items()}
    loss(leaf).backward()
    for k in P:
        d = torch.randn(P[k].shape, generator=torch.Generator().manual_seed(5)).cuda()
        d = d / d.norm()  # a unit step: second-order terms stay small
        eps = 1e-2
        num = (loss(dict(P, **{k: P[k] + eps * d})) - loss(dict(P, **{k: P[k] - eps * d}))) / (2 * eps)
        ana = (leaf[k].grad.double() * d).sum()
        assert (num - ana).abs() <= 1e-2 * max(1.0, ana.abs().item()), (k, num.item(), ana.item())


@pytest.mark.parametrize("B,T", [(0, 5), (0, 4096), (3, 0)])
def test_nothing_to_do(B, T):
    """No sequences, or sequences without tokens: empty outputs, zero parameter gradients, states handed on."""
    C = 24
    x = torch.zeros(B, T, C, device="cuda", dtype=BF)
    w, b, st = torch.ones(C, 4, device="cuda"), torch.ones(C, device="cuda"), torch.ones(B, 3, C, device="cuda", dtype=BF)
    y, last = gdr.conv_forward(x, w, b, st, output_final_state=True)
    dx, dw, db, ds = gdr.conv_backward(x, w, b, x, st, st)
    assert y.shape == dx.shape == x.shape and torch.equal(last, st) and torch.equal(ds, st) and not dw.any() and not db.any()
    A, S0 = -torch.ones(C, 16, device="cuda"), torch.ones(B, C, 16, device="cuda")
    bc = torch.zeros(B, T, 1, 16, device="cuda", dtype=BF)
    y, S_T, saved = gdr.ssm_forward(x, x, A, bc, bc, b, b, S0)
    dx, ddt, dA, dB, dC, dD, dbias, dS0 = gdr.ssm_backward(x, x, A, bc, bc, saved, x, b, b, S0)
    assert torch.equal(S_T, S0) and torch.equal(dS0, S0) and not dA.any() and not dD.any() and not dbias.any()
    r, y = gdr.norm_forward(x, b, x, b, x, b)
    g = gdr.norm_backward(x, b, x, b, r, b, x, x)
    assert r.shape == y.shape == x.shape and not g[3].any() and not g[4].any() and not g[5].any()


@pytest.mark.parametrize("B", [1, 3])
def test_gradients_broadcast_over_tokens(B):
    """The gradient of a mean over tokens comes as one row repeated (token stride 0): as if it were written out."""
    r = gen(31)
    T, C, N = 37, 24, 8
    x, w, dt, z = r(B, T, C).cuda(), r(C, 4).cuda(), r(B, T, C, mul=0.3).cuda(), r(B, T, C).cuda()
    A, Bm, Cm, wt = -torch.exp(r(C, N)).cuda(), r(B, T, 1, N).cuda(), r(B, T, 1, N).cuda(), r(C).cuda()
    row = r(B, C).cuda()

    def grads(f, shape_of_dy, *leaves):
        ls = [t.clone().requires_grad_() for t in leaves]
        return torch.autograd.grad(f(*ls), ls, shape_of_dy)

    for f, leaves in ((lambda a, b: gdr.causal_conv(a, b)[0], (x, w)),
                      (lambda a, b, c, d, e: gdr.selective_scan(a, b, c, d, e)[0], (x, dt, A, Bm, Cm)),
                      (lambda a, b, c: gdr.block_norm(a, b, c)[0], (x, wt, z))):
        dy = row[:, None].expand(B, T, C)
        for a, b in zip(grads(f, dy, *leaves), grads(f, dy.contiguous(), *leaves)):
            assert torch.equal(a, b)


def test_plain_norm_of_a_slice_has_a_gradient():
    r = gen(33)
    big, w, dy = r(7, 48).cuda(), r(16).cuda(), r(7, 16).cuda()

    def grads(x):
        x, v = x.detach().requires_grad_(), w.clone().requires_grad_()
        return torch.autograd.grad(gdr.block_norm(x, pre_weight=v)[1], (x, v), dy)

    for a, b in zip(grads(big[:, 16:32]), grads(big[:, 16:32].contiguous())):
        assert torch.equal(a, b)


def test_packed_tokens_beyond_32_bit_offsets():
    """The last sequence of a packed batch whose elements lie past 2^31: as the sequence alone."""
    r = gen(41)
    C, N, lens = 2048, 4, [1 << 20, 37]
    T, n = sum(lens), lens[1]

    def tail(*shape, mul=1.0):
        t = torch.zeros(1, T, *shape, dtype=BF, device="cuda")
        t[:, -n:] = r(1, n, *shape, dtype=BF, mul=mul).cuda()
        return t

    cu = cu_of(lens).cuda()
    x, dy, dt, Bm, Cm = tail(C), tail(C), tail(C, mul=0.5), tail(1, N), tail(1, N)
    w, A, b = r(C, 4).cuda(), -torch.exp(r(C, N)).cuda(), r(C).cuda()

    def last(t):
        return t[:, -n:].contiguous()

    y, _ = gdr.conv_forward(x, w, b, None, cu)
    dx = gdr.conv_backward(x, w, b, dy, None, None, cu)[0]
    assert torch.equal(last(y), gdr.conv_forward(last(x), w, b)[0])
    assert torch.equal(last(dx), gdr.conv_backward(last(x), w, b, last(dy))[0])
    del y, dx
    y, S, saved = gdr.ssm_forward(x, dt, A, Bm, Cm, b, None, None, cu)
    g = gdr.ssm_backward(x, dt, A, Bm, Cm, saved, dy, b, None, None, cu)
    y1, S1, saved1 = gdr.ssm_forward(last(x), last(dt), A, last(Bm), last(Cm), b)
    g1 = gdr.ssm_backward(last(x), last(dt), A, last(Bm), last(Cm), saved1, last(dy), b)
    assert torch.equal(last(y), y1) and torch.equal(S[1:], S1)
    for i in (0, 1, 3, 4):
        assert torch.equal(last(g[i]), g1[i]), i
    del y, S, saved, g
    out = gdr.norm_forward(x, b, dy)[0]
    assert torch.equal(last(out), gdr.norm_forward(last(x), b, last(dy))[0])
    d, d1 = gdr.norm_backward(x, b, dy, dr=dt), gdr.norm_backward(last(x), b, last(dy), dr=last(dt))
    assert torch.equal(last(d[0]), d1[0]) and torch.equal(last(d[1]), d1[1])


def test_pools_beyond_32_bit_offsets():
    """A slot whose state lies past 2^31 elements of the pool: as in a pool of one."""
    r = gen(42)
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both(state, call):  # state: [1, ...]; the call's outputs and the states after it
        at = (1 << 31) // state[0].numel() + 1
        pool = torch.empty(at + 1, *state.shape[1:], dtype=state.dtype, device="cuda")
        pool[at] = state[0]
        one = state.clone()
        assert torch.equal(call(pool, slot + at), call(one, slot))
        assert torch.equal(pool[at], one[0])

    x, w = r(1, 2048, dtype=BF).cuda(), r(2048, 4).cuda()
    both(r(1, 3, 2048, dtype=BF).cuda(), lambda p, s: gdr.conv_step(x, p, w, None, s))
    A, bc = -torch.exp(r(2048, 16)).cuda(), r(1, 1, 16, dtype=BF).cuda()
    both(r(1, 2048, 16).cuda(), lambda p, s: gdr.ssm_step(x, x, A, bc, bc, p, None, None, s))
    q, g, beta = r(1, 2, 128, dtype=BF).cuda(), -r(1, 2).abs().cuda(), torch.sigmoid(r(1, 2, dtype=BF)).cuda()
    for layout in ("KV", "VK"):
        both(r(1, 2, 128, 128).cuda(), lambda p, s: gdr.step(q, q, q, g, beta, p, layout, None, s, gdr.GDR_PROLOGUE_QK_L2NORM))
