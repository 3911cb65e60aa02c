"""Cases for the operators around the gated delta rule: the short causal convolution, the selective
state space scan, the block norms and the single-token step.

With ``own`` false, ``run`` evaluates an operator in plain torch (32 bits throughout, rounded once
at the end); with ``own`` true it makes the calls of ``chunked_gated_delta_04_gb300`` that a user
makes.  ``exact`` evaluates the definitions in 64 bits, token by token.

  conv  pre[t] = b + sum_j w[j] X[t - (W-1) + j] over the sequence's tokens X preceded by W-1 rows of
        state; y = silu(pre) or pre
  ssm   a_t = exp(D_t A), h_t = a_t h_{t-1} + D_t x_t B_t, y_t = sum_n C_t h_t + D x_t,
        D_t = softplus(dt_t + dt_bias)
  norm  u = x [rstd(x) w_post] [silu(z)] [scale]; r = [residual +] u; y = r rstd(r) w_pre
  step  S = e^g S (I - beta k k^T) + beta v k^T, o = S q / sqrt(DK), one token per sequence

Every case names its own sizes; ``lens`` lists the sequence lengths of a packed batch (empty: ``B``
sequences of ``T`` tokens).
"""
import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"


def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _lens(case):
    if case.get("lens"):
        return [int(v) for v in case["lens"].split(",")]
    return [case["T"]] * case["B"]


# ------------------------------------------------------------------------------------- the cases
def listed():
    eight = "6291,877,3530,256,8192,1999,5004,2431"  # eight prompts of 256 to 8192 tokens
    return [
        # decode: one token of one sequence through the convolution of q, k and v (16 heads of 128 each)
        dict(name="conv_step_b1", op="conv", way="step", dtype=BF16, B=1, slots=4, C=6144, W=4, act="silu", bias=False),
        # prompts of eight users in one packed batch, each going on from its own state
        dict(name="conv_prompt_varlen8", op="conv", way="fwd", dtype=BF16, B=1, T=0, lens=eight, C=2048, W=4, act="silu",
             bias=True, state=True),
        # a training step's convolution at the benchmark's B = 2, T = 4096, q, k and v in one tensor
        dict(name="conv_train_b2_t4096", op="conv", way="train", dtype=BF16, B=2, T=4096, lens="", C=6144, W=4, act="silu",
             bias=False, state=False),
        # decode: 64 sequences of a served batch, one token each
        dict(name="ssm_step_b64", op="ssm", way="step", dtype=BF16, B=64, slots=80, D=4096, N=16, G=1),
        # packed prompts in fp32, states handed to decoding, nothing kept for a backward; an odd length and a one-token one
        dict(name="ssm_prompt_fp32", op="ssm", way="fwd", dtype=F32, B=1, T=0, lens="1025,1,2048,577", D=1536, N=16, G=1,
             state=True),
        # one long prompt: few channels, so the sequence itself has to be split
        dict(name="ssm_prompt_t32768", op="ssm", way="fwd", dtype=BF16, B=1, T=32768, lens="", D=1024, N=16, G=1, state=False),
        # a training step at B = 2, T = 4096: outputs and every gradient
        dict(name="ssm_train_b2_t4096", op="ssm", way="train", dtype=BF16, B=2, T=4096, lens="", D=4096, N=16, G=1, state=True),
        # decode: residual add and norm in front of the next block, 32 rows
        dict(name="norm_add_rows32", op="norm", way="fwd", mode="add", dtype=BF16, res=BF16, rows=32, D=2048),
        # the gated norm of a mixer's output per head, trained: 2 x 4096 tokens, 16 heads of 128
        dict(name="norm_gated_train", op="norm", way="train", mode="gated", dtype=BF16, res=BF16, rows=131072, D=128),
        # norms on both sides of a block with gate, residual scale and an fp32 residual stream: the backward
        dict(name="norm_full_bwd", op="norm", way="bwd", mode="full", dtype=BF16, res=F32, rows=8192, D=4096),
        # decode: one sequence, 16 heads, inputs raw (normalised and mapped inside)
        dict(name="step_b1", op="step", way="step", dtype=BF16, B=1, slots=1, Hk=16, Hv=16, DK=128, DV=128, layout="KV",
             raw=True),
        # decode: a served batch with grouped value heads, states in a pool
        dict(name="step_b128_grouped", op="step", way="step", dtype=BF16, B=128, slots=160, Hk=16, Hv=32, DK=128, DV=128,
             layout="VK", raw=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _packing(rng, case, total):
    """Either B sequences of T tokens or a packed batch whose lengths differ widely (one may be empty)."""
    n = rng.choice([1, 1, 2, 3, 5, 8])
    case.update(B=n, T=max(1, total // n), lens="")
    if rng.random() < 0.5:
        parts = [rng.random() ** 2 for _ in range(n)]
        lens = [int(total * v / sum(parts)) for v in parts]
        lens[rng.randrange(n)] += 1
        case.update(B=1, T=0, lens=",".join(str(v) for v in lens))


def _draw_any(rng):
    op = rng.choice(["conv", "ssm", "norm", "step"])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "conv":
        case = dict(op=op, way=rng.choice(["fwd", "train", "step"]), dtype=dtype, C=_log(rng, 64, 8192), W=rng.choice([2, 3, 4]),
                    act=rng.choice(["silu", "none"]), bias=rng.random() < 0.5)
        if rng.random() < 0.7:
            case["C"] = max(64, case["C"] // 64 * 64)
        if case["way"] == "step":
            case.update(B=_log(rng, 1, 256))
            case.update(slots=case["B"] + rng.randrange(0, 8))
        else:
            case.update(state=rng.random() < 0.5)
            _packing(rng, case, _log(rng, 1, 33000))
    elif op == "ssm":
        G = rng.choice([1, 1, 2, 4])
        case = dict(op=op, way=rng.choice(["fwd", "train", "step"]), dtype=dtype, D=G * _log(rng, 16, 6144 // G),
                    N=rng.choice([4, 8, 16, 16, 32, 64]), G=G)
        if rng.random() < 0.7:
            case["D"] = max(64, case["D"] // 64 * 64)
        if case["way"] == "step":
            case.update(B=_log(rng, 1, 256))
            case.update(slots=case["B"] + rng.randrange(0, 8))
        else:
            case.update(state=rng.random() < 0.5)
            _packing(rng, case, _log(rng, 1, 33000))
    elif op == "norm":
        mode = rng.choice(["add", "gated", "full"])
        way = rng.choice(["fwd", "bwd", "train"]) if mode == "gated" else rng.choice(["fwd", "bwd"])
        D = rng.choice([64, 128, 96, 256]) if mode == "gated" else _log(rng, 64, 8192)
        if mode != "gated" and rng.random() < 0.7:
            D = max(64, D // 64 * 64)
        case = dict(op=op, way=way, mode=mode, dtype=dtype, res=F32 if mode == "full" or dtype == F32 else BF16,
                    rows=_log(rng, 1, (1 << 25) // D), D=D)
    else:
        Hk = rng.choice([1, 2, 4, 8, 16])
        case = dict(op=op, way="step", dtype=dtype, B=_log(rng, 1, 256), Hk=Hk, Hv=Hk * rng.choice([1, 1, 2, 3]),
                    DK=rng.choice([16, 64, 80, 128, 128]), DV=rng.choice([16, 64, 96, 128, 128]),
                    layout=rng.choice(["KV", "VK"]), raw=rng.random() < 0.5)
        case.update(slots=case["B"] + rng.randrange(0, 8))
    return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {}
    for c in listed():
        key = (c["op"], c["way"] == "step")
        most[key] = max(most.get(key, 0), _cost(c))
    while True:
        case = _draw_any(rng)
        if _cost(case) <= most[(case["op"], case["way"] == "step")]:
            return case


# ------------------------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _dt(case)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def uni(*shape):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["way"] == "step":
        # the batch's states lie anywhere in the pool
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:case["B"]].to(torch.int32)
    elif case["op"] != "norm":
        lens = _lens(case)
        s["lens"] = lens
        s["cu"] = None
        if case["lens"]:
            s["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        B, T = (1, sum(lens)) if case["lens"] else (case["B"], case["T"])
        M = len(lens)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        s["w"] = rand(C, W) * (1.0 / math.sqrt(W))
        s["b"] = rand(C) * 0.1 if case["bias"] else None
        if case["way"] == "step":
            s["x"] = rand(case["B"], C).to(dt)
            s["state"] = rand(case["slots"], W - 1, C).to(dt)
        else:
            s["x"] = rand(B, T, C).to(dt)
            s["state"] = rand(M, W - 1, C).to(dt) if case["state"] else None
            if case["way"] == "train":
                s["dy"] = rand(B, T, C).to(dt)
                s["dstate"] = rand(M, W - 1, C).to(dt) if case["state"] else None
    elif case["op"] == "ssm":
        D, N, G = case["D"], case["N"], case["G"]
        lead = (case["B"],) if case["way"] == "step" else (B, T)
        s["x"] = rand(*lead, D).to(dt)
        s["dt"] = (rand(*lead, D) * 0.5).to(dt)
        s["Bm"] = rand(*lead, G, N).to(dt)
        s["Cm"] = rand(*lead, G, N).to(dt)
        # decay rates 1 .. N per state; steps of 1e-3 to 1e-1 after the softplus
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32).expand(D, N) * torch.exp(0.1 * rand(D, N))
        step = torch.exp(uni(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["Dskip"] = 1.0 + 0.1 * rand(D)
        if case["way"] == "step":
            s["state"] = rand(case["slots"], D, N) * 0.3
        else:
            s["S0"] = rand(M, D, N) * 0.3 if case["state"] else None
            if case["way"] == "train":
                s["dy"] = rand(B, T, D).to(dt)
                s["dS_T"] = rand(M, D, N) * 0.1 if case["state"] else None
    elif case["op"] == "norm":
        R, D = case["rows"], case["D"]
        res = torch.bfloat16 if case["res"] == BF16 else torch.float32
        add, full = case["mode"] == "add", case["mode"] == "full"
        s["x"] = rand(R, D).to(dt)
        s["z"] = None if add else rand(R, D).to(dt)
        s["w_post"] = None if add else 1.0 + 0.1 * rand(D)
        s["w_pre"] = 1.0 + 0.1 * rand(D) if add or full else None
        s["scale"] = 0.2 + 0.05 * rand(D) if full else None
        s["residual"] = rand(R, D).to(res) if add or full else None
        if case["way"] != "fwd":
            s["dy"] = rand(R, D).to(dt)  # gradient of the normed output (of the only output when there is no stream)
            s["dr"] = rand(R, D).to(res) if add or full else None
            s["r"] = rand(R, D).to(res) if add or full else None  # the stream as the forward stored it
    else:
        Bn, Hk, Hv, DK, DV = (case[k] for k in ("B", "Hk", "Hv", "DK", "DV"))
        q, k = rand(Bn, Hk, DK), rand(Bn, Hk, DK)
        a, b = rand(Bn, Hv), rand(Bn, Hv)
        if not case["raw"]:
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
            a, b = torch.log(torch.sigmoid(a)), torch.sigmoid(b)
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), rand(Bn, Hv, DV).to(dt)
        s["g"], s["beta"] = a, b.to(dt)
        s["state"] = rand(case["slots"], Hv, *((DK, DV) if case["layout"] == "KV" else (DV, DK))) * 0.3
    return s


# --------------------------------------------------------------------------------- the framework
def _run_own(s):
    import chunked_gated_delta_04_gb300 as gdr

    case = s["case"]
    op, way = case["op"], case["way"]
    if op == "conv":
        if way == "step":
            y = gdr.conv_step(s["x"], s["state"], s["w"], s["b"], slots=s["slots"], activation=case["act"])
            return {"y": y, "state": s["state"]}
        y, last = gdr.conv_forward(s["x"], s["w"], s["b"], s["state"], s["cu"], activation=case["act"], output_final_state=True)
        out = {"y": y, "last": last}
        if way == "train":
            dx, dw, db, dstate = gdr.conv_backward(s["x"], s["w"], s["b"], s["dy"], s["state"], s["dstate"], s["cu"],
                                                   activation=case["act"])
            out.update(dx=dx, dw=dw, db=db, dstate=dstate)
        return out
    if op == "ssm":
        if way == "step":
            y = gdr.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], s["Dskip"], s["dt_bias"], slots=s["slots"])
            return {"y": y, "state": s["state"]}
        y, last, saved = gdr.ssm_forward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["Dskip"], s["dt_bias"], s["S0"], s["cu"],
                                         save=way == "train")
        out = {"y": y, "last": last}
        if way == "train":
            names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dS0")
            grads = gdr.ssm_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], saved, s["dy"], s["Dskip"], s["dt_bias"],
                                     s["dS_T"], s["cu"], want_dS0=s["S0"] is not None)
            out.update(zip(names, grads))
        return out
    if op == "norm":
        out = {}
        if way != "bwd":
            r, y = gdr.norm_forward(s["x"], s["w_post"], s["z"], s["scale"], s["residual"], s["w_pre"])
            out.update(r=r, y=y)
        if way != "fwd":
            gated = case["mode"] == "gated"
            names = ("dx", "dz", "dresidual", "dw_post", "dscale", "dw_pre")
            grads = gdr.norm_backward(s["x"], s["w_post"], s["z"], s["scale"], s["r"], s["w_pre"],
                                      dr=s["dy"] if gated else s["dr"], dy=None if gated else s["dy"])
            out.update(zip(names, grads))
        return out
    o = gdr.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], layout=case["layout"], slots=s["slots"],
                 prologue=gdr.GDR_PROLOGUE_ALL if case["raw"] else 0)
    return {"o": o, "state": s["state"]}


# ------------------------------------------------------------------------------- the plain forms
def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _starts(s):
    """Per sequence its first token and its end, and per token its sequence."""
    lens = torch.tensor(s["lens"], dtype=torch.int64, device=s["x"].device)
    end = torch.cumsum(lens, 0)
    return end - lens, end, torch.repeat_interleave(torch.arange(len(s["lens"]), device=end.device), lens)


def _conv_plain(s):
    case = s["case"]
    W, C, dt = case["W"], case["C"], s["x"].dtype
    w, silu = s["w"], case["act"] == "silu"
    bias = s["b"] if s["b"] is not None else torch.zeros_like(w[:, 0])
    if case["way"] == "step":
        at = s["slots"].long()
        win = torch.cat([s["state"][at], s["x"][:, None]], 1).float()
        pre = (win * w.t()).sum(1) + bias
        s["state"][at] = win[:, 1:].to(dt)
        return {"y": (pre * _sigmoid(pre) if silu else pre).to(dt), "state": s["state"]}
    x = s["x"].reshape(-1, C).float()
    first, end, seq = _starts(s)
    # every sequence with W-1 rows of state in front of it
    place = torch.arange(x.shape[0], device=x.device) + (seq + 1) * (W - 1)
    tail = (end + torch.arange(len(s["lens"]), device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    head = tail - (end - first)[:, None]
    padded = x.new_zeros(x.shape[0] + len(s["lens"]) * (W - 1), C)
    padded[place] = x
    if s["state"] is not None:
        padded[head] = s["state"].float()
    pre = bias.expand(x.shape[0], C)
    for j in range(W):
        pre = pre + padded[place - (W - 1) + j] * w[:, j]
    gate = _sigmoid(pre)
    out = {"y": (pre * gate if silu else pre).to(dt).reshape(s["x"].shape), "last": padded[tail].to(dt)}
    if case["way"] == "train":
        dpre = s["dy"].reshape(-1, C).float()
        if silu:
            dpre = dpre * (gate + pre * gate * (1 - gate))
        dpadded = torch.zeros_like(padded)
        if s["dstate"] is not None:
            dpadded[tail] = s["dstate"].float()
        dw = []
        for j in range(W):
            rows = place - (W - 1) + j
            dw.append((dpre * padded[rows]).sum(0))
            dpadded[rows] += dpre * w[:, j]
        out.update(dx=dpadded[place].to(dt).reshape(s["x"].shape), dw=torch.stack(dw, 1), db=dpre.sum(0) if s["b"] is not None else None,
                   dstate=dpadded[head].to(dt) if s["state"] is not None else None)
    return out


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis (h before the first: 0), by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]]) if 2 * step < a.shape[0] else a
        step *= 2
    return b


def _ssm_plain(s):
    case = s["case"]
    D, N, G, dt = case["D"], case["N"], case["G"], s["x"].dtype
    x, raw = s["x"].reshape(-1, D).float(), s["dt"].reshape(-1, D).float() + s["dt_bias"]
    delta = _softplus(raw)
    Bm, Cm = (s[k].reshape(-1, G, 1, N).float() for k in ("Bm", "Cm"))
    M = x.shape[0]

    def spread(v):  # [tokens, G, 1, N] as [tokens, D, N]
        return v.expand(M, G, D // G, N).reshape(M, D, N)

    if case["way"] == "step":
        at = s["slots"].long()
        h = s["state"][at] * torch.exp(delta[..., None] * s["A"]) + (delta * x)[..., None] * spread(Bm)
        s["state"][at] = h
        return {"y": ((h * spread(Cm)).sum(-1) + s["Dskip"] * x).to(dt), "state": s["state"]}
    first, end, seq = _starts(s)
    some = (end > first).nonzero()[:, 0]
    head, tail = first[some], end[some] - 1
    decay = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * spread(Bm)
    inner = decay.clone()
    inner[head] = 0.0
    if s["S0"] is not None:
        b[head] += decay[head] * s["S0"][some]
    h = _scan(inner, b)
    del b
    last = s["S0"].clone() if s["S0"] is not None else torch.zeros(len(s["lens"]), D, N, device=x.device)
    last[some] = h[tail]
    y = (h * spread(Cm)).sum(-1) + s["Dskip"] * x
    out = {"y": y.to(dt).reshape(s["x"].shape), "last": last}
    if case["way"] == "train":
        dy = s["dy"].reshape(-1, D).float()
        dh = dy[..., None] * spread(Cm)
        if s["dS_T"] is not None:
            dh[tail] += s["dS_T"][some]
        # the same scan in reverse: dh_t takes a_{t+1} dh_{t+1}, nothing across a sequence's end
        dh = _scan(torch.cat([inner[1:], torch.zeros_like(inner[:1])]).flip(0), dh.flip(0)).flip(0)
        del inner
        before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
        before[head] = s["S0"][some] if s["S0"] is not None else 0.0
        dC = (dy[..., None] * h).reshape(M, G, D // G, N).sum(2)
        del h
        dlog = dh * decay * before
        del before
        dhB = (dh * spread(Bm)).sum(-1)
        dB = (dh * (delta * x)[..., None]).reshape(M, G, D // G, N).sum(2)
        ddelta = (dlog * s["A"]).sum(-1) + dhB * x
        ddt = ddelta * _sigmoid(raw)
        dS0 = None
        if s["S0"] is not None:
            dS0 = s["dS_T"].clone()
            dS0[some] = decay[head] * dh[head]
        shape = s["x"].shape
        out.update(dx=(dhB * delta + s["Dskip"] * dy).to(dt).reshape(shape), ddt=ddt.to(dt).reshape(shape),
                   dA=(dlog * delta[..., None]).sum(0), dB=dB.to(dt).reshape(s["Bm"].shape), dC=dC.to(dt).reshape(s["Cm"].shape),
                   dD=(dy * x).sum(0), ddt_bias=ddt.sum(0), dS0=dS0)
    return out


def _rstd(v, eps=1e-6):
    return (v.square().mean(-1, keepdim=True) + eps).rsqrt()


def _norm_plain(s):
    case = s["case"]
    x, dt = s["x"].float(), s["x"].dtype
    zg = _sigmoid(s["z"].float()) if s["z"] is not None else None
    act = s["z"].float() * zg if s["z"] is not None else 1.0
    wp = s["w_post"] if s["w_post"] is not None else 1.0
    sc = s["scale"] if s["scale"] is not None else 1.0
    xh = x * _rstd(x) if s["w_post"] is not None else x
    out = {}
    if case["way"] != "bwd":
        r = xh * wp * act * sc
        if s["residual"] is not None:
            r = r + s["residual"].float()
        r = r.to(s["residual"].dtype if s["residual"] is not None else dt)
        rf = r.float()
        out.update(r=r, y=(rf * _rstd(rf) * s["w_pre"]).to(dt) if s["w_pre"] is not None else None)
    if case["way"] != "fwd":
        names = ("dx", "dz", "dresidual", "dw_post", "dscale", "dw_pre")
        g = dict.fromkeys(names)
        dy = s["dy"].float()
        if s["w_pre"] is not None:
            r = s["r"].float()
            rs = _rstd(r)
            rh = r * rs
            g["dw_pre"] = (dy * rh).sum(0)
            t = dy * s["w_pre"]
            du = s["dr"].float() + rs * (t - rh * (t * rh).mean(-1, keepdim=True))
            g["dresidual"] = du.to(s["r"].dtype)
        else:
            du = dy
        if s["scale"] is not None:
            g["dscale"] = (du * xh * wp * act).sum(0)
        if s["z"] is not None:
            g["dz"] = (du * sc * xh * wp * (zg + act * (1 - zg))).to(dt)
        t = du * sc * act
        if s["w_post"] is not None:
            g["dw_post"] = (t * xh).sum(0)
            t = t * wp
            t = _rstd(x) * (t - xh * (t * xh).mean(-1, keepdim=True))
        g["dx"] = t.to(dt)
        out.update(g)
    return out


def _step_plain(s):
    case = s["case"]
    rep = case["Hv"] // case["Hk"]
    q, k, v, beta, g = s["q"].float(), s["k"].float(), s["v"].float(), s["beta"].float(), s["g"]
    if case["raw"]:
        q = q * (q.square().sum(-1, keepdim=True) + 1e-6).rsqrt()
        k = k * (k.square().sum(-1, keepdim=True) + 1e-6).rsqrt()
        g, beta = -_softplus(-g), _sigmoid(beta)
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    at = s["slots"].long()
    S = s["state"][at]
    S = (S.transpose(-1, -2) if case["layout"] == "KV" else S) * torch.exp(g)[..., None, None]
    miss = v - (S * k[:, :, None]).sum(-1)
    S = S + (beta[..., None] * miss)[..., None] * k[:, :, None]
    o = (S * q[:, :, None]).sum(-1) * (1.0 / math.sqrt(case["DK"]))
    s["state"][at] = S.transpose(-1, -2) if case["layout"] == "KV" else S
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


_PLAIN = {"conv": _conv_plain, "ssm": _ssm_plain, "norm": _norm_plain, "step": _step_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------- work
def work(case):
    el = 2 if case["dtype"] == BF16 else 4
    op, way = case["op"], case["way"]
    if op == "conv":
        C, W = case["C"], case["W"]
        if way == "step":
            n = case["B"] * C
            return {"bytes": n * el * (2 + 2 * (W - 1)) + 4 * C * W, "flops": 2 * W * n}
        lens = _lens(case)
        n, st = sum(lens) * C, len(lens) * (W - 1) * C
        passes, taps = (2, 1) if way == "fwd" else (4, 3)  # train: x, y, dy, dx
        states = (2 if case["state"] else 1) * (1 if way == "fwd" else 2)
        return {"bytes": el * (passes * n + states * st) + 4 * C * W * (1 if way == "fwd" else 2), "flops": 2 * W * n * taps}
    if op == "ssm":
        D, N, G = case["D"], case["N"], case["G"]
        tokens = case["B"] if way == "step" else sum(_lens(case))
        if way == "step":
            return {"bytes": el * (3 * tokens * D + 2 * tokens * G * N) + 8 * tokens * D * N + 4 * D * N, "flops": 7 * tokens * D * N}
        states = len(_lens(case)) * D * N
        if way == "fwd":
            return {"bytes": el * (3 * tokens * D + 2 * tokens * G * N) + 4 * states * (1 + case["state"]) + 4 * D * N,
                    "flops": 7 * tokens * D * N}
        return {"bytes": el * (6 * tokens * D + 4 * tokens * G * N) + 4 * states * (1 + 3 * case["state"]) + 8 * D * N,
                "flops": 26 * tokens * D * N}
    if op == "norm":
        n, rl = case["rows"] * case["D"], 2 if case["res"] == BF16 else 4
        add, gated = case["mode"] == "add", case["mode"] == "gated"
        fwd = el * (2 if add else 3) + (0 if gated else 2 * rl)  # x [z] [residual] -> [r] y
        bwd = el * 5 if gated else el * (2 if add else 5) + 3 * rl  # x z dy [dr r] -> dx dz [dresidual]
        return {"bytes": n * {"fwd": fwd, "bwd": bwd, "train": fwd + bwd}[way], "flops": n * {"fwd": 10, "bwd": 25, "train": 35}[way]}
    n = case["B"] * case["Hv"]
    return {"bytes": 8 * n * case["DK"] * case["DV"] + el * (2 * case["B"] * case["Hk"] * case["DK"] + 2 * n * case["DV"] + n) + 4 * n,
            "flops": 7 * n * case["DK"] * case["DV"]}


# ------------------------------------------------------------------------------------- in 64 bits
def _exact_conv(s, case):
    W, w, x = case["W"], s["w"].double(), s["x"].double()
    silu = case["act"] == "silu"
    bias = s["b"].double() if s["b"] is not None else torch.zeros(case["C"], dtype=torch.float64, device=x.device)
    if case["way"] == "step":
        at = s["slots"].long()
        old = s["state"].double()
        new = old.clone()
        pre = bias + w[:, W - 1] * x
        for j in range(W - 1):
            pre = pre + w[:, j] * old[at, j]
            new[at, j] = old[at, j + 1] if j + 2 < W else x
        return {"y": pre / (1 + torch.exp(-pre)) if silu else pre, "state": new}
    flat = x.reshape(-1, case["C"])
    ys, lasts, dxs, dstates, t0 = [], [], [], [], 0
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    dy = s["dy"].double().reshape(-1, case["C"]) if case["way"] == "train" else None
    for n, L in enumerate(s["lens"]):
        state = s["state"][n].double() if s["state"] is not None else flat.new_zeros(W - 1, case["C"])
        X = torch.cat([state, flat[t0:t0 + L]])
        pre = sum((X[j:j + L] * w[:, j] for j in range(W)), bias.expand(L, -1))
        sg = 1 / (1 + torch.exp(-pre))
        ys.append(pre * sg if silu else pre)
        lasts.append(X[L:])
        if dy is not None:
            d = dy[t0:t0 + L] * (sg * (1 + pre * (1 - sg)) if silu else 1.0)
            dX = torch.zeros_like(X)
            if s["dstate"] is not None:
                dX[L:] += s["dstate"][n].double()
            for j in range(W):
                dX[j:j + L] += d * w[:, j]
                dw[:, j] += (d * X[j:j + L]).sum(0)
            db += d.sum(0)
            dxs.append(dX[W - 1:])
            dstates.append(dX[:W - 1])
        t0 += L
    out = {"y": torch.cat(ys).reshape(x.shape), "last": torch.stack(lasts)}
    if dy is not None:
        out.update(dx=torch.cat(dxs).reshape(x.shape), dw=dw, db=db if s["b"] is not None else None,
                   dstate=torch.stack(dstates) if s["state"] is not None else None)
    return out


def _exact_ssm(s, case):
    D, N, G = case["D"], case["N"], case["G"]
    flat = {k: s[k].double().reshape(-1, D) for k in ("x", "dt")}
    x, raw = flat["x"], flat["dt"] + s["dt_bias"].double()
    delta = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    A, skip = s["A"].double(), s["Dskip"].double()
    group = torch.arange(D, device=x.device) // (D // G)
    Bm, Cm = (s[k].double().reshape(-1, G, N) for k in ("Bm", "Cm"))
    if case["way"] == "step":
        at = s["slots"].long()
        state = s["state"].double()
        h = torch.exp(delta[..., None] * A) * state[at] + (delta * x)[..., None] * Bm[:, group]
        state[at] = h
        return {"y": torch.einsum("bdn,bdn->bd", h, Cm[:, group]) + skip * x, "state": state}
    lens = s["lens"]
    first = [sum(lens[:n]) for n in range(len(lens))]
    last = s["S0"].double() if s["S0"] is not None else torch.zeros(len(lens), D, N, dtype=torch.float64, device=x.device)
    train = case["way"] == "train"
    y = torch.empty_like(x)
    before = torch.empty(x.shape[0], D, N, dtype=torch.float64, device=x.device) if train else None
    # the sequences side by side, longest first: at token t the ones still running are a prefix
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    h = last[order].clone()
    starts = torch.tensor([first[n] for n in order], device=x.device)
    running = [sum(lens[n] > t for n in order) for t in range(max(lens))]
    for t, m in enumerate(running):
        at = starts[:m] + t
        if train:
            before[at] = h[:m]
        h[:m] = torch.exp(delta[at][..., None] * A) * h[:m] + (delta[at] * x[at])[..., None] * Bm[at][:, group]
        y[at] = (h[:m] * Cm[at][:, group]).sum(-1) + skip * x[at]
    last = torch.empty_like(h)
    last[order] = h
    out = {"y": y.reshape(s["x"].shape), "last": last}
    if train:
        dy = s["dy"].double().reshape(-1, D)
        dh = s["dS_T"].double()[order] if s["dS_T"] is not None else torch.zeros_like(h)
        dA = torch.zeros_like(A)
        dx, ddelta, dB, dC = torch.empty_like(x), torch.empty_like(x), torch.empty_like(Bm), torch.empty_like(Cm)
        for t in reversed(range(len(running))):
            m = running[t]
            at = starts[:m] + t
            a, was, ex = torch.exp(delta[at][..., None] * A), before[at], (delta[at] * x[at])[..., None]
            here = a * was + ex * Bm[at][:, group]
            d = dh[:m] + dy[at][..., None] * Cm[at][:, group]
            dC[at] = (dy[at][..., None] * here).reshape(m, G, D // G, N).sum(2)
            dB[at] = (d * ex).reshape(m, G, D // G, N).sum(2)
            dlog = d * a * was
            dA += (dlog * delta[at][..., None]).sum(0)
            into = (d * Bm[at][:, group]).sum(-1)
            dx[at] = into * delta[at] + skip * dy[at]
            ddelta[at] = (dlog * A).sum(-1) + into * x[at]
            dh[:m] = a * d
        ddt = ddelta / (1 + torch.exp(-raw))
        dS0 = torch.empty_like(dh)
        dS0[order] = dh
        out.update(dx=dx.reshape(s["x"].shape), ddt=ddt.reshape(s["x"].shape), dA=dA, dB=dB.reshape(s["Bm"].shape),
                   dC=dC.reshape(s["Cm"].shape), dD=(dy * x).sum(0), ddt_bias=ddt.sum(0), dS0=dS0 if s["S0"] is not None else None)
    return out


def _exact_norm(s, case):
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    leaf = {k: f[k].requires_grad_() for k in ("x", "z", "w_post", "scale", "w_pre") if f[k] is not None}

    def rms(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)

    u = rms(leaf["x"]) * leaf["w_post"] if f["w_post"] is not None else leaf["x"]
    if f["z"] is not None:
        u = u * leaf["z"] / (1 + torch.exp(-leaf["z"]))
    if f["scale"] is not None:
        u = u * leaf["scale"]
    out = {}
    if case["way"] != "bwd":
        r = (u if f["residual"] is None else u + f["residual"]).detach()
        y = None
        if f["w_pre"] is not None:
            stored = r.to(s["residual"].dtype).double()
            y = (rms(stored) * f["w_pre"]).detach()
        out.update(r=r, y=y)
    if case["way"] != "fwd":
        out.update(dict.fromkeys(("dx", "dz", "dresidual", "dw_post", "dscale", "dw_pre")))
        du = f["dy"]
        if f["w_pre"] is not None:
            r = f["r"].detach().requires_grad_()
            dr, out["dw_pre"] = torch.autograd.grad((rms(r) * leaf["w_pre"] * f["dy"]).sum(), [r, leaf["w_pre"]])
            du = out["dresidual"] = f["dr"] + dr
        wanted = [k for k in ("x", "z", "w_post", "scale") if k in leaf]
        for k, v in zip(wanted, torch.autograd.grad((u * du).sum(), [leaf[k] for k in wanted])):
            out["d" + k] = v
    return out


def _exact_step(s, case):
    rep = case["Hv"] // case["Hk"]
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    if case["raw"]:
        q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        g, beta = torch.nn.functional.logsigmoid(g), torch.sigmoid(beta)
    state = s["state"].double()
    at = s["slots"].long()
    kv = case["layout"] == "KV"
    S = state[at].transpose(-1, -2) if kv else state[at]
    head = torch.arange(case["Hv"], device=q.device) // rep
    k, q = k[:, head], q[:, head]
    S = torch.exp(g)[..., None, None] * (S - torch.einsum("bh,bhv,bhk->bhvk", beta, torch.einsum("bhvk,bhk->bhv", S, k), k)) \
        + torch.einsum("bh,bhv,bhk->bhvk", beta, v, k)
    state[at] = S.transpose(-1, -2).contiguous() if kv else S
    return {"o": torch.einsum("bhvk,bhk->bhv", S, q) / math.sqrt(case["DK"]), "state": state}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ssm" and case["way"] != "step" and max(_lens(case)) > 40000:
        return None
    return {"conv": _exact_conv, "ssm": _exact_ssm, "norm": _exact_norm, "step": _exact_step}[case["op"]](s, case)
