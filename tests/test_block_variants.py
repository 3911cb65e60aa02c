"""Variants that sizes choose, against the fp64 references: sequences of equal length cut into segments, steps with
four rows per thread; which outputs there are.  Inputs, comparison and tolerances (sequences of up to ~300 tokens) are
those of test_block.py."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from oracle import block as ob
from test_block import BF, F32, check, conv_inputs, cu_of, gen, norm_inputs, npy, ssm_inputs, ssm_ref, ssm_run, wide

pytestmark = pytest.mark.gpu
SMS = 152


# ------------------------------------------------------------------------------- selective scan
def batch(d, B, T):
    """ssm_inputs' packed tensors as B sequences of T tokens."""
    return {k: v.reshape(B, T, *v.shape[2:]) if v is not None and v.shape[:2] == (1, B * T) else v for k, v in d.items()}


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,D,N,G,state,strided,soft", [
    (2, 300, 200, 16, 1, True, False, True),
    (3, 321, 64, 8, 1, False, False, True),
    (2, 257, 72, 32, 2, True, True, True),     # a last segment of one token, groups, slices of wider tensors
    (1, 300, 130, 4, 1, True, False, False),
    (3, 130, 36, 64, 4, True, True, True),     # channels of a group that do not divide by four
    (2, 128, 65, 16, 1, False, True, True),    # whole segments, element-wise rows
])
def test_ssm_equal_lengths_cut_into_segments(dtype, B, T, D, N, G, state, strided, soft):
    lens = [T] * B
    d = ssm_inputs(dtype, D, N, G, lens, state)
    if not soft:
        d["dt"] = d["dt"].abs() * 0.1
        d["dt_bias"] = None
    ref = ssm_ref(d, lens, soft)
    d = batch(d, B, T)
    if strided:
        d.update({k: wide(d[k], 5, 2) for k in ("x", "dt", "dy")})
    units = B * -(-T // 64)  # segments have 64 tokens here: their boundary states are in the workspace
    assert gdr.ssm_workspace(d["x"], d["Bm"]).numel() > units * D * N * 4 > 256
    check(ssm_run(d, None, soft), ref)


def test_ssm_packed_segments_equal_the_sequences_alone():
    lens = [500, 64, 1, 333]
    d = ssm_inputs(F32, 96, 16, 1, lens, True)
    packed = ssm_run(d, cu_of(lens).cuda())
    sums = dict.fromkeys(("dA", "dD", "ddt_bias"), 0)
    at = 0
    for n, L in enumerate(lens):
        one = {k: v[:, at:at + L].contiguous() if v.shape[:2] == (1, sum(lens)) else v[n:n + 1] if k in ("S0", "dS_T") else v
               for k, v in d.items()}
        alone = ssm_run(one, None)
        check({k: packed[k][:, at:at + L] for k in ("y", "dx", "ddt", "dB", "dC")}, {k: npy(alone[k]) for k in ("y", "dx", "ddt", "dB", "dC")})
        check({k: packed[k][n:n + 1] for k in ("S_T", "dS0")}, {k: npy(alone[k]) for k in ("S_T", "dS0")})
        for k in sums:
            sums[k] = sums[k] + npy(alone[k])
        at += L
    check({k: packed[k] for k in sums}, sums)


# -------------------------------------------------------------------- steps, four rows per thread
def some_slots(B, pool, seed):
    """Rows anywhere in the pool; of every seventh the slot is outside it."""
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))[:B].to(torch.int32)
    slots[3::14], slots[10::14] = -1, pool
    return slots


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("C,W,B,strided", [(4096, 4, 307, False), (4096, 2, 306, True), (1023, 3, 305, False)])
def test_conv_step_of_many_rows(dtype, C, W, B, strided):
    lanes = C // 4 if C % 4 == 0 else C
    assert -(-lanes // 256) * -(-B // 4) >= 2 * SMS and B % 4
    r = gen(B)
    x, w, b, pool = r(B, C, dtype=dtype).cuda(), r(C, W, mul=0.5).cuda(), r(C).cuda(), r(B + 9, W - 1, C, dtype=dtype).cuda()
    if strided:
        x = wide(x[:, None], 8, 4)[:, 0]
    slots, before = some_slots(B, B + 9, 1), pool.clone()
    y = gdr.conv_step(x, pool, w, b, slots.cuda())
    live = (slots >= 0) & (slots < B + 9)
    rows, at = live.nonzero()[:, 0].cuda(), slots[live].long().cuda()
    ref = ob.conv(npy(x[rows]), npy(w), npy(b), npy(before[at]), [1] * len(rows))
    check(dict(y=y[rows], last=pool[at]), ref)
    assert not y[(~live).cuda()].any()
    rest = torch.ones(B + 9, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,N,G,B", [(4096, 16, 1, 63), (2050, 4, 2, 289), (1040, 64, 4, 41)])
def test_ssm_step_of_many_rows(dtype, D, N, G, B):
    assert -(-D * N // 4 // 256) * -(-B // 4) >= 4 * SMS and B % 4
    d = ssm_inputs(dtype, D, N, G, [B], False)
    x, dt, Bm, Cm = (d[k][0] for k in ("x", "dt", "Bm", "Cm"))
    pool = gen(9)(B + 9, D, N).cuda()
    slots, before = some_slots(B, B + 9, 2), pool.clone()
    y = gdr.ssm_step(x, dt, d["A"], Bm, Cm, pool, d["D"], d["dt_bias"], slots.cuda())
    live = (slots >= 0) & (slots < B + 9)
    rows, at = live.nonzero()[:, 0].cuda(), slots[live].long().cuda()
    ref = ob.ssm(*(npy(t) for t in (x[rows], dt[rows], d["A"], Bm[rows], Cm[rows], d["D"], d["dt_bias"], before[at])), [1] * len(rows))
    check(dict(y=y[rows], S_T=pool[at]), ref)
    assert not y[(~live).cuda()].any()
    rest = torch.ones(B + 9, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(pool[rest], before[rest])


# ------------------------------------------------------------------------------ which outputs
def there(outputs, wanted):
    assert [t is not None for t in outputs] == [bool(v) for v in wanted]


@pytest.mark.parametrize("absent", [None, "b", "state"])
def test_conv_outputs(absent):
    d = conv_inputs(BF, 16, 4, [5, 3], True, True)
    if absent is not None:
        d[absent] = None
    cu = cu_of([5, 3]).cuda()
    for final in (False, True):
        there(gdr.conv_forward(d["x"], d["w"], d["b"], d["state"], cu, output_final_state=final), (1, final))
    there(gdr.conv_backward(d["x"], d["w"], d["b"], d["dy"], d["state"], d["dl"], cu), (1, 1, absent != "b", absent != "state"))


@pytest.mark.parametrize("absent", [None, "D", "dt_bias", "S0", "dS_T"])
def test_ssm_outputs(absent):
    d = ssm_inputs(BF, 16, 8, 1, [5, 3], True)
    if absent is not None:
        d[absent] = None
    cu = cu_of([5, 3]).cuda()
    args = [d[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    for final in (False, True):
        for save in (False, True):
            out = gdr.ssm_forward(*args, d["D"], d["dt_bias"], d["S0"], cu, True, final, save)
            there(out, (1, final, save))
    for want in (False, True):
        there(gdr.ssm_backward(*args, out[2], d["dy"], d["D"], d["dt_bias"], d["dS_T"], cu, want_dS0=want),
              (1, 1, 1, 1, 1, absent != "D", absent != "dt_bias", want))


@pytest.mark.parametrize("mode", ["gated", "add", "full", "plain", "post", "stream", "scale"])
def test_norm_outputs(mode):
    d = norm_inputs(mode, F32, F32, (5, 48))
    has = {k: v is not None for k, v in d.items()}
    r, y = gdr.norm_forward(d["x"], d["post"], d["z"], d["scale"], d["res"], d["pre"])
    there((r, y), (has["res"] or not has["pre"], has["pre"]))
    there(gdr.norm_backward(d["x"], d["post"], d["z"], d["scale"], r if has["res"] else None, d["pre"], d["dr"], d["dy"]),
          (1, has["z"], has["res"], has["post"], has["scale"], has["pre"]))


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32)])
def test_norm_backward_of_one_output(types):
    """Of two outputs either gradient may be absent: as one of zeros."""
    d = norm_inputs("full", *types, (5, 48))
    r, _ = gdr.norm_forward(d["x"], d["post"], d["z"], d["scale"], d["res"], d["pre"])

    def grads(dr, dy):
        return gdr.norm_backward(d["x"], d["post"], d["z"], d["scale"], r, d["pre"], dr, dy)

    for a, b in ((grads(d["dr"], None), grads(d["dr"], torch.zeros_like(d["dy"]))), (grads(None, d["dy"]), grads(torch.zeros_like(d["dr"]), d["dy"]))):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
