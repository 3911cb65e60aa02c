"""Cases for the attention mixer that stands beside the delta rule in a hybrid model: rotary positions,
attention (forward and backward), the single-token step over a paged cache, and the write of a prompt
into that cache.

With ``own`` false, ``run`` evaluates an operator in plain torch (32 bits, angles in 64, rounded once at
the end); with ``own`` true it makes the calls of ``chunked_gated_delta_04_gb300`` that a user makes.
``exact`` evaluates the definitions in 64 bits.

  rope   (y_a, y_b) = scale * (x_a cos t - x_b sin t, x_b cos t + x_a sin t), t = position * freq_i, for
         the pairs (i, i + R/2) or (2i, 2i + 1) of the first R features of a head; the others are passed on
  attn   p_ij = softmax over the visible j of scale q_i.k_j, o_i = sum_j p_ij v_j, lse_i = log sum exp;
         with n queries and m keys, query i sees the keys j <= i + m - n (causal) that are above
         i + m - n - window (window > 0); a query that sees none has o = 0 and lse = -infinity
  step   one token per row: k, v go to position lengths[b] of the row's pages, then the token attends to
         positions 0 .. lengths[b]
  write  k, v of prompts into their rows' pages, from position starts[n] on

``lens`` lists the sequence lengths of a packed batch (empty: ``B`` sequences of ``T`` tokens); ``more`` keys
stand in front of a sequence's own (an earlier part of the prompt).
"""
import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"


def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _ints(text):
    return [int(v) for v in text.split(",")]


def _lens(case):
    return _ints(case["lens"]) if case.get("lens") else [case["T"]] * case["B"]


# ------------------------------------------------------------------------------------- the cases
def listed():
    eight = "6291,877,3530,256,8192,1999,5004,2431"  # eight prompts of 256 to 8192 tokens
    return [
        # decode: 64 sequences, one token each, somewhere in contexts of up to 65536 tokens
        dict(name="rope_step_b64", op="rope", way="step", dtype=BF16, B=64, T=1, lens="", Hq=16, Hk=4, D=128, R=128,
             pairs="half", scaled=False),
        # a training step at the benchmark's B = 2, T = 4096: a rotation of half of each head and its gradient
        dict(name="rope_train_b2_t4096", op="rope", way="train", dtype=BF16, B=2, T=4096, lens="", Hq=16, Hk=16, D=128, R=64,
             pairs="half", scaled=False),
        # packed prompts in fp32, frequencies scaled for a context longer than the trained one, neighbouring pairs
        dict(name="rope_prompt_fp32", op="rope", way="fwd", dtype=F32, B=1, T=0, lens="1025,1,2048,577", Hq=16, Hk=4, D=80, R=80,
             pairs="neighbours", scaled=True),
        # prompts of eight users in one packed batch, key heads shared by four query heads
        dict(name="attn_prompt_varlen8", op="attn", way="fwd", dtype=BF16, B=1, T=0, lens=eight, more=0, Hq=16, Hk=4, D=128,
             causal=True, window=0),
        # the next part of three prompts behind 2816 tokens each, sliding window
        dict(name="attn_prompt_window", op="attn", way="fwd", dtype=BF16, B=3, T=515, lens="", more=2816, Hq=8, Hk=8, D=64,
             causal=True, window=1024),
        # a training step's attention at the benchmark's B = 2, T = 4096, H = 16, D = 128
        dict(name="attn_train_b2_t4096", op="attn", way="train", dtype=BF16, B=2, T=4096, lens="", more=0, Hq=16, Hk=16, D=128,
             causal=True, window=0),
        # the same for one longer sequence with shared key heads
        dict(name="attn_train_t8192", op="attn", way="train", dtype=BF16, B=1, T=8192, lens="", more=0, Hq=32, Hk=8, D=128,
             causal=True, window=0),
        # training in fp32 on a packed batch of ragged lengths
        dict(name="attn_train_fp32", op="attn", way="train", dtype=F32, B=1, T=0, lens="577,1,1025,300", more=0, Hq=4, Hk=2, D=64,
             causal=True, window=0),
        # decode: one sequence of 65536 tokens, so that its cache has to be split
        dict(name="attn_step_t65536", op="step", way="step", dtype=BF16, lens="65535", page=64, spare=16, Hq=16, Hk=4, D=128,
             window=0),
        # decode: 64 sequences of one token to 8192
        dict(name="attn_step_b64", op="step", way="step", dtype=BF16, lens=",".join(str(i * i * 8191 // 3969) for i in range(64)),
             page=64, spare=64, Hq=32, Hk=8, D=128, window=0),
        # a short prompt of one user goes to its pages
        dict(name="cache_write_one", op="write", way="fwd", dtype=BF16, lens="256", start=0, page=64, spare=16, Hk=4, D=128),
        # eight users' prompts go to their pages, behind a part of 100 tokens written before
        dict(name="cache_write_varlen8", op="write", way="fwd", dtype=BF16, lens=eight, start=100, page=64, spare=64, Hk=8, D=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut(rng, total, n):
    parts = [rng.random() ** 2 + 1e-3 for _ in range(n)]
    return ",".join(str(max(1, int(total * v / sum(parts)))) for v in parts)


def _packing(rng, case, total):
    """Either B sequences of T tokens or a packed batch whose lengths differ widely."""
    n = rng.choice([1, 1, 2, 3, 5, 8])
    case.update(B=n, T=max(1, total // n), lens="")
    if rng.random() < 0.5:
        case.update(B=1, T=0, lens=_cut(rng, max(n, total), n))


def _draw_any(rng):
    op = rng.choice(["rope", "attn", "attn", "step", "write"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    D = rng.choice([64, 128, 128, 80, 96, 32])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 4, 5, 8])
    if op == "rope":
        case = dict(op=op, way=rng.choice(["fwd", "train", "step"]), dtype=dtype, Hq=Hq, Hk=Hk, D=D,
                    R=rng.choice([D, D, D // 2, D - 10]), pairs=rng.choice(["half", "neighbours"]), scaled=rng.random() < 0.4)
        if case["way"] == "step":
            case.update(B=_log(rng, 1, 256), T=1, lens="")
        else:
            _packing(rng, case, _log(rng, 1, 33000))
    elif op == "attn":
        case = dict(op=op, way=rng.choice(["fwd", "train"]), dtype=dtype, Hq=Hq, Hk=Hk, D=D, causal=rng.random() < 0.8)
        # training sequences of a few tokens have gradients that are nothing but rounding (of one token: zero)
        _packing(rng, case, _log(rng, 1 if case["way"] == "fwd" else 256, 12000 if dtype == BF16 else 3000))
        case.update(more=rng.choice([0, 0, 0, _log(rng, 1, 3000)]) if case["way"] == "fwd" else 0,
                    window=rng.choice([0, 0, 0, _log(rng, 16, 4000)]))
    elif op == "step":
        n, longest = _log(rng, 1, 200), _log(rng, 1, 66000)
        case = dict(op=op, way="step", dtype=dtype, lens=",".join(str(rng.randrange(longest)) for _ in range(n)),
                    page=rng.choice([16, 32, 64, 64, 128]), spare=rng.randrange(64), Hq=Hq, Hk=Hk, D=D,
                    window=rng.choice([0, 0, 0, _log(rng, 16, 8000)]))
    else:
        n = rng.choice([1, 2, 3, 5, 8])
        case = dict(op=op, way="fwd", dtype=dtype, lens=_cut(rng, max(n, _log(rng, 1, 33000)), n), start=rng.randrange(300),
                    page=rng.choice([16, 32, 64, 64, 128]), spare=rng.randrange(64), Hk=Hk, D=D)
    return case


def _cost(case):
    """A pass's cost in bytes: products in fp32 are worth more of them than those in bf16.  A window makes it no cheaper, nor
    do narrow heads: the plain forms hold whole rows of probabilities and of the cache."""
    w = work({**case, "window": 0})
    flops = w["flops"] * 128 / case["D"] if case["op"] == "attn" else w["flops"]
    return max(w["bytes"], flops / (10 if case["dtype"] == F32 else 200))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"], c["way"]] = max(most.get((c["op"], c["way"]), 0), _cost(c))
    while True:
        case = _draw_any(rng)
        if _cost(case) <= most[case["op"], case["way"]]:
            return case


# ------------------------------------------------------------------------------------ the inputs
def _frequencies(R, scaled):
    """Radians per position of the R / 2 pairs, base 10000, and the factor of the rotation.  Scaled for 16 times a trained
    context of 4096: pairs that turn over 32 times in it stay, those that turn less than once are slowed 16-fold, those
    between are mixed, and the rotation grows by 0.1 ln 16 + 1."""
    half = torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R
    freq = 10000.0 ** -half
    if not scaled:
        return freq, 1.0
    turns = 4096 * freq / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return freq * keep + freq / 16 * (1 - keep), 0.1 * math.log(16) + 1


def _pages(s, case, lengths, gen):
    """Block tables of rows that hold `lengths` tokens, their pages anywhere in the pool, -1 behind them."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    free = torch.randperm(sum(need) + case["spare"], generator=gen, device="cuda").to(torch.int32)
    wide = torch.arange(max(need), device="cuda")
    count = torch.tensor(need, device="cuda")
    at = (torch.cumsum(count, 0) - count)[:, None] + wide
    s["table"] = torch.where(wide < count[:, None], free[at.clamp(max=free.numel() - 1)], -1).to(torch.int32).contiguous()
    return free.numel()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = _dt(case), case["op"]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": case}
    lens = _lens(case)
    s["lens"] = lens

    def cu(lengths):
        return torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()

    if op in ("rope", "attn"):
        packed = bool(case["lens"])
        B, T = (1, sum(lens)) if packed else (case["B"], case["T"])
        s["cu"] = cu(lens) if packed else None
    if op == "rope":
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        # q and k as they lie in one projection's output, beside v
        lead = (B,) if case["way"] == "step" else (B, T)
        qkv = rand(*lead, Hq + 2 * Hk, D)
        s["q"], s["k"] = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hk, :]
        s["freqs"], s["scale"] = _frequencies(case["R"], case["scaled"])
        s["positions"] = None  # the tokens' places in their sequences
        if case["way"] == "step" or case["scaled"]:  # contexts that go on
            s["positions"] = torch.randint(0, 65536, lead, generator=gen, device="cuda").to(torch.int32)
        if case["way"] == "train":
            s["dq"], s["dk"] = rand(*lead, Hq, D), rand(*lead, Hk, D)
    elif op == "attn":
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        s["keys"] = [n + case["more"] for n in lens]
        Tk = sum(s["keys"]) if packed else T + case["more"]
        s["cu_k"] = cu(s["keys"]) if packed and case["more"] else s["cu"]
        s["q"], s["k"], s["v"] = rand(B, T, Hq, D), rand(B, Tk, Hk, D), rand(B, Tk, Hk, D)
        if case["way"] == "train":
            s["do"] = rand(B, T, Hq, D)
    elif op == "step":
        n = len(lens)
        s["lengths"] = torch.tensor(lens, dtype=torch.int32).cuda()
        pages = _pages(s, case, [v + 1 for v in lens], gen)
        s["q"], s["k"], s["v"] = rand(n, case["Hq"], case["D"]), rand(n, case["Hk"], case["D"]), rand(n, case["Hk"], case["D"])
        s["k_cache"], s["v_cache"] = (rand(pages, case["page"], case["Hk"], case["D"]) for _ in range(2))
    else:
        s["cu"] = cu(lens)
        s["starts"] = torch.full((len(lens),), case["start"], dtype=torch.int32, device="cuda")
        pages = _pages(s, case, [v + case["start"] for v in lens], gen)
        s["k"], s["v"] = rand(1, sum(lens), case["Hk"], case["D"]), rand(1, sum(lens), case["Hk"], case["D"])
        s["k_cache"], s["v_cache"] = (rand(pages, case["page"], case["Hk"], case["D"]) for _ in range(2))
    return s


# --------------------------------------------------------------------------------- the framework
def _run_own(s):
    import chunked_gated_delta_04_gb300 as gdr

    case = s["case"]
    op = case["op"]
    if op == "rope":
        how = dict(positions=s["positions"], cu_seqlens=s["cu"], interleaved=case["pairs"] == "neighbours", scale=s["scale"])
        q, k = gdr.rope_forward(s["q"], s["k"], s["freqs"], **how)
        out = {"q": q, "k": k}
        if case["way"] == "train":
            out["dq"], out["dk"] = gdr.rope_backward(s["dq"], s["dk"], s["freqs"], **how)
        return out
    if op == "attn":
        how = dict(cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"], causal=case["causal"], window=case["window"])
        o, lse = gdr.attn_forward(s["q"], s["k"], s["v"], **how)
        out = {"o": o, "lse": lse}
        if case["way"] == "train":
            out["dq"], out["dk"], out["dv"] = gdr.attn_backward(s["q"], s["k"], s["v"], o, lse, s["do"], **how)
        return out
    if op == "step":
        o = gdr.attn_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], window=case["window"])
        return {"o": o, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    gdr.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], starts=s["starts"], cu_seqlens=s["cu"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------------------------------- the plain forms
def _places(s):
    """Of every token its place in its sequence and its sequence."""
    lens = torch.tensor(s["lens"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device="cuda"), lens)
    return torch.arange(seq.numel(), device="cuda") - (torch.cumsum(lens, 0) - lens)[seq], seq


def _turned(x, cos, sin, R, neighbours):
    v = x.float()
    a, b = (v[..., 0:R:2], v[..., 1:R:2]) if neighbours else (v[..., :R // 2], v[..., R // 2:R])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).flatten(-2) if neighbours else torch.cat([ya, yb], -1)
    return torch.cat([y.to(x.dtype), x[..., R:]], -1)


def _rope_plain(s):
    case = s["case"]
    at = s["positions"] if s["positions"] is not None else _places(s)[0].reshape(s["q"].shape[:-2])
    angle = at.double()[..., None, None] * s["freqs"]
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    how = case["R"], case["pairs"] == "neighbours"
    out = {"q": _turned(s["q"], cos, sin, *how), "k": _turned(s["k"], cos, sin, *how)}
    if case["way"] == "train":
        out.update(dq=_turned(s["dq"], cos, -sin, *how), dk=_turned(s["dk"], cos, -sin, *how))
    return out


def _attn_heads(q, k, v, do, case):
    """Attention of [batch, heads, tokens, features] in 32 bits; k and v of one head for every G of q."""
    B, Hq, n, D = q.shape
    Hk, m = k.shape[1:3]
    G, scale = Hq // Hk, 1.0 / math.sqrt(D)
    q = q.reshape(B, Hk, G * n, D).float()
    k, v = k.float(), v.float()
    s = (q @ k.transpose(-1, -2)).view(B, Hk, G, n, m) * scale
    if case["causal"] or case["window"]:
        i = torch.arange(n, device=q.device)[:, None] + (m - n)
        j = torch.arange(m, device=q.device)
        hidden = torch.zeros(n, m, dtype=torch.bool, device=q.device)
        if case["causal"]:
            hidden = j > i
        if case["window"]:
            hidden = hidden | (j <= i - case["window"])
        s.masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    s.div_(torch.where(total == 0, 1.0, total))
    lse = (torch.log(total) + top).view(B, Hq, n)
    p = s.view(B, Hk, G * n, m)
    o = p @ v
    grads = None
    if do is not None:
        do = do.reshape(B, Hk, G * n, D).float()
        dv = p.transpose(-1, -2) @ do
        ds = do @ v.transpose(-1, -2)
        ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        grads = (ds @ k).view(B, Hq, n, D), ds.transpose(-1, -2) @ q, dv
    return o.view(B, Hq, n, D), lse, grads


def _attn_plain(s):
    case, dt = s["case"], s["q"].dtype

    def heads(t):
        return t.transpose(1, 2)

    if s["cu"] is None:
        parts = [_attn_heads(heads(s["q"]), heads(s["k"]), heads(s["v"]), heads(s["do"]) if "do" in s else None, case)]
    else:  # the sequences of a packed batch are of unlike lengths: one after the other
        q, k, v = (t.split(n, 1) for t, n in ((s["q"], s["lens"]), (s["k"], s["keys"]), (s["v"], s["keys"])))
        do = s["do"].split(s["lens"], 1) if "do" in s else [None] * len(q)
        parts = [_attn_heads(heads(a), heads(b), heads(c), heads(d) if d is not None else None, case) for a, b, c, d in zip(q, k, v, do)]

    def whole(ts):
        return torch.cat([heads(t) for t in ts], 1).to(dt).contiguous()

    out = {"o": whole([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts], -1)}
    if case["way"] == "train":
        out.update((name, whole([p[2][i] for p in parts])) for i, name in enumerate(("dq", "dk", "dv")))
    return out


def _at(s, rows, places):
    """Pages and places in them of the rows' positions."""
    page = s["case"]["page"]
    return s["table"][rows, places // page].long(), places % page


def _step_plain(s):
    case = s["case"]
    n, Hk, D = s["k"].shape
    lengths = s["lengths"].long()
    rows = torch.arange(n, device="cuda")
    page, slot = _at(s, rows, lengths)
    s["k_cache"][page, slot], s["v_cache"][page, slot] = s["k"], s["v"]
    # the rows' pages side by side, as long as the longest row; what is behind a row's end is hidden
    pages = s["table"].long().clamp(min=0)
    k, v = (s[name][pages].flatten(1, 2) for name in ("k_cache", "v_cache"))
    at = torch.arange(k.shape[1], device="cuda")
    seen = at <= lengths[:, None]
    if case["window"]:
        seen = seen & (at > lengths[:, None] - case["window"])
    q = s["q"].float().view(n, Hk, -1, D)
    sc = q @ k.float().permute(0, 2, 3, 1) * (1.0 / math.sqrt(D))
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = (p / p.sum(-1, keepdim=True)) @ v.float().masked_fill(~seen[..., None, None], 0.0).transpose(1, 2)
    return {"o": o.reshape(s["q"].shape).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _write_plain(s):
    place, seq = _places(s)
    page, slot = _at(s, seq, place + s["starts"].long()[seq])
    s["k_cache"][page, slot], s["v_cache"][page, slot] = s["k"][0], s["v"][0]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


_PLAIN = {"rope": _rope_plain, "attn": _attn_plain, "step": _step_plain, "write": _write_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------- work
def _pairs(n, m, causal, window):
    """Pairs of a query and a key that it sees."""
    i = torch.arange(n) + (m - n)
    last = i.clamp(max=m - 1) if causal else torch.full_like(i, m - 1)
    first = (i - window + 1).clamp(min=0) if window else torch.zeros_like(i)
    return int((last - first + 1).clamp(min=0).sum())


def work(case):
    el, op = (2 if case["dtype"] == BF16 else 4), case["op"]
    lens = _lens(case)
    Hk, D = case["Hk"], case["D"]
    if op == "rope":
        n = sum(lens) * (case["Hq"] + Hk) * (2 if case["way"] == "train" else 1)
        return {"bytes": 2 * el * n * D, "flops": 3 * n * case["R"]}
    if op == "attn":
        Hq, keys = case["Hq"], [n + case["more"] for n in lens]
        pairs = Hq * sum(_pairs(n, m, case["causal"], case["window"]) for n, m in zip(lens, keys))
        q, k, train = el * sum(lens) * Hq * D, el * sum(keys) * Hk * D, case["way"] == "train"
        return {"bytes": (4 * q + 4 * k if train else 2 * q + 2 * k) + 4 * sum(lens) * Hq, "flops": (14 if train else 4) * pairs * D}
    if op == "step":
        seen = sum(min(n + 1, case["window"] or n + 1) for n in lens)
        return {"bytes": el * D * (2 * seen * Hk + 2 * len(lens) * (case["Hq"] + Hk)), "flops": 4 * seen * case["Hq"] * D}
    return {"bytes": 4 * el * sum(lens) * Hk * D, "flops": 0}


# ------------------------------------------------------------------------------------- in 64 bits
def _exact_rope(s, case):
    spots = s["positions"]
    if spots is None:
        spots = torch.cat([torch.arange(n, device="cuda") for n in s["lens"]]).view(s["q"].shape[:-2])
    turn = torch.polar(torch.full_like(s["freqs"], s["scale"]).expand(*spots.shape, -1), spots.double().unsqueeze(-1) * s["freqs"])
    R = case["R"]

    def rotate(x, by):
        y = x.double().clone()
        first = torch.arange(R // 2, device="cuda") * (2 if case["pairs"] == "neighbours" else 1)
        second = first + (1 if case["pairs"] == "neighbours" else R // 2)
        z = torch.complex(y[..., first], y[..., second]) * by.unsqueeze(-2)
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": rotate(s["q"], turn), "k": rotate(s["k"], turn)}
    if case["way"] == "train":
        out.update(dq=rotate(s["dq"], turn.conj()), dk=rotate(s["dk"], turn.conj()))
    return out


def _exact_attn(s, case):
    q, k, v = (s[name].double() for name in ("q", "k", "v"))
    B, T, Hq, D = q.shape
    G, train = Hq // k.shape[2], case["way"] == "train"
    o, lse = torch.zeros_like(q), torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    spans, a, b = [], 0, 0  # (batch row, first query, queries, first key, keys)
    for i, (n, m) in enumerate(zip(s["lens"], s["keys"])):
        spans.append((0, a, n, b, m) if s["cu"] is not None else (i, 0, n, 0, m))
        a, b = a + n, b + m
    for row, q0, n, k0, m in spans:
        for h in range(Hq):
            kk, vv = k[row, k0:k0 + m, h // G], v[row, k0:k0 + m, h // G]
            for t in range(0, n, 1024):
                e = min(n, t + 1024)
                i = torch.arange(t, e, device=q.device) + (m - n)
                lo = max(0, t + m - n - case["window"] + 1) if case["window"] else 0
                hi = max(0, min(m, e + m - n)) if case["causal"] else m
                if hi <= lo:
                    continue
                j = torch.arange(lo, hi, device=q.device)
                see = torch.ones(e - t, hi - lo, dtype=torch.bool, device=q.device)
                if case["causal"]:
                    see &= j[None] <= i[:, None]
                if case["window"]:
                    see &= j[None] > i[:, None] - case["window"]
                qq = q[row, q0 + t:q0 + e, h]
                z = torch.where(see, torch.einsum("id,jd->ij", qq, kk[lo:hi]) / math.sqrt(D), -math.inf)
                ls = torch.logsumexp(z, -1)
                p = torch.where(see, torch.exp(z - ls[:, None]), 0.0)
                out = torch.einsum("ij,jd->id", p, vv[lo:hi])
                lse[row, h, q0 + t:q0 + e], o[row, q0 + t:q0 + e, h] = ls, out
                if train:
                    g = s["do"][row, q0 + t:q0 + e, h].double()
                    dv[row, k0 + lo:k0 + hi, h // G] += torch.einsum("ij,id->jd", p, g)
                    dz = p * (torch.einsum("id,jd->ij", g, vv[lo:hi]) - (g * out).sum(-1)[:, None]) / math.sqrt(D)
                    dq[row, q0 + t:q0 + e, h] = torch.einsum("ij,jd->id", dz, kk[lo:hi])
                    dk[row, k0 + lo:k0 + hi, h // G] += torch.einsum("ij,id->jd", dz, qq)
    out = {"o": o, "lse": lse}
    if train:
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def _exact_step(s, case):
    kc, vc, o, page = s["k_cache"].double(), s["v_cache"].double(), s["q"].double().clone(), case["page"]
    G = case["Hq"] // case["Hk"]
    for b, n in enumerate(s["lens"]):
        last = int(s["table"][b, n // page])
        kc[last, n % page], vc[last, n % page] = s["k"][b].double(), s["v"][b].double()
        mine = s["table"][b, :n // page + 1].long()
        first = max(0, n + 1 - case["window"]) if case["window"] else 0
        k, v = (c[mine].reshape(-1, case["Hk"], case["D"])[first:n + 1].repeat_interleave(G, 1) for c in (kc, vc))
        w = torch.softmax(torch.einsum("hd,jhd->hj", s["q"][b].double(), k) / math.sqrt(case["D"]), -1)
        o[b] = torch.einsum("hj,jhd->hd", w, v)
    return {"o": o, "k_cache": kc, "v_cache": vc}


def _exact_write(s, case):
    kc, vc, t = s["k_cache"].double(), s["v_cache"].double(), 0
    for n, L in enumerate(s["lens"]):
        pos = torch.arange(case["start"], case["start"] + L, device="cuda")
        flat = s["table"][n].long()[pos // case["page"]] * case["page"] + pos % case["page"]
        kc.view(-1, case["Hk"], case["D"])[flat] = s["k"][0, t:t + L].double()
        vc.view(-1, case["Hk"], case["D"])[flat] = s["v"][0, t:t + L].double()
        t += L
    return {"k_cache": kc, "v_cache": vc}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "step": _exact_step, "write": _exact_write}[case["op"]](s, case)
