"""The precision of the gated delta rule's float32 and bfloat16 results on the GPU, head by head (bfloat16
results all heads together), against the float64 form (oracle/sublayer_ops.py); tolerances and inputs in delta_precision.py."""
import numpy as np
import pytest

import delta_precision as D
from hc_testutil import have_gpu, note
from oracle import sublayer_ops as R

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc


def put(a, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16 if dt == "bf16" else torch.float32)


def get(t):
    return t.detach().double().cpu().numpy()


def device(ins, dt):
    """(q, k, v, g, beta, state, do, dstate) on the GPU."""
    return [put(a, dt if i in (0, 1, 2, 6) else "f32") for i, a in enumerate(ins)]


def check(name, where, x, y, dt, tol):
    """x against y: float32 to `tol`, bfloat16 against the rounded y."""
    if dt == "bf16":
        y = D.bf16(y)
        tol = D.half(y)
    off = D.rel(x, y)
    assert off <= tol, (name, where, off, tol)


def check_forward(o, M, ins, dt, lengths=None, grow=1.0):
    B, S, _, Dk = ins[0].shape
    ro, rM = R.gated_delta(*ins[:6], lengths)
    o, M = get(o), get(M)
    if dt == "bf16":
        check("o", "all", o, ro, dt, None)
    for b in range(B):
        n = S if lengths is None else lengths[b]
        for h in range(ins[2].shape[2]):
            if n and dt == "f32":
                check("o", (b, h), o[b, :n, h], ro[b, :n, h], dt, D.OUT * grow)
            check("state", (b, h), M[b, h], rM[b, h], "f32", D.STATE * grow)


# B, S, Hk, Hv, Dk, Dv of every width's variants, in one walk
SIZES = [(1, 300, 1, 2, 64, 48), (4, 500, 2, 4, 128, 128), (1, 900, 1, 1, 72, 100), (1, 200, 2, 2, 256, 64),
         (1, 330, 1, 2, 100, 36), (1, 130, 1, 1, 200, 30)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward(size, dt):
    note(f"precision of hc_gated_delta {size} {dt}")
    ins = D.inputs(*size, dt, sum(size))
    d = device(ins, dt)
    o, M = hc.hc_gated_delta(*d[:6])
    torch.cuda.synchronize()
    check_forward(o, M, ins, dt)


def check_backward(got, ins, dt, lengths=None, grow=1.0):
    B, S, Hk, _ = ins[0].shape
    ref = R.gated_delta_backward(*ins[:5], ins[6], ins[5], ins[7], lengths)
    got = [get(t) for t in got]
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate0"), got, ref):
        if dt == "bf16" and name in ("dq", "dk", "dv"):
            check(name, "all", x, y, dt, None)
            continue
        tol = (D.DG if name == "dg" else D.OUT) * grow
        for b in range(B):
            for h in range(y.shape[1 if name == "dstate0" else 2]):
                u, v = (x[b, h], y[b, h]) if name == "dstate0" else (x[b, :, h], y[b, :, h])
                if name == "dg" and np.any(v) and D.rel(u, v) > tol:  # of states' products that cancel
                    n = S if lengths is None else lengths[b]
                    check(name, (b, h), u, v, "f32", tol * max(1.0, D.dg_size(ins, n, b, h) / np.linalg.norm(v)))
                elif np.any(v):
                    check(name, (b, h), u, v, "f32", tol)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward(size, dt):
    note(f"precision of hc_gated_delta_backward {size} {dt}")
    ins = D.inputs(*size, dt, sum(size))
    d = device(ins, dt)
    got = hc.hc_gated_delta_backward(*d[:5], d[6], d[5], d[7])
    torch.cuda.synchronize()
    check_backward(got, ins, dt)


# few heads and long sequences, which are walked in segments: an odd and an even number of them, the last one
# short or whole, every width's variants; `slow` decays carry the first state through all of them
SEGMENTS = [(1, 1100, 1, 2, 128, 128), (1, 2100, 1, 1, 64, 32), (1, 1300, 1, 1, 256, 48), (1, 2048, 1, 2, 100, 40),
            (1, 8192, 1, 1, 128, 16)]


@pytest.mark.parametrize("size", SEGMENTS)
@pytest.mark.parametrize("slow", [None, 1e-4, 1e-5, 0.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_segments_forward(size, slow, dt):
    note(f"precision of hc_gated_delta {size} {dt} slow={slow}")
    ins = D.inputs(*size, dt, sum(size), slow)
    d = device(ins, dt)
    o, M = hc.hc_gated_delta(*d[:6])
    state = d[5].clone()
    o2, M2 = hc.hc_gated_delta(*d[:5], state, out=(None, state))
    torch.cuda.synchronize()
    check_forward(o, M, ins, dt, grow=D.joins(size[1]))
    assert torch.equal(o, o2) and torch.equal(M, M2)


@pytest.mark.parametrize("size", SEGMENTS)
@pytest.mark.parametrize("slow", [None, 1e-4, 0.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_segments_backward(size, slow, dt):
    note(f"precision of hc_gated_delta_backward {size} {dt} slow={slow}")
    ins = D.inputs(*size, dt, sum(size), slow)
    d = device(ins, dt)
    got = hc.hc_gated_delta_backward(*d[:5], d[6], d[5], d[7])
    torch.cuda.synchronize()
    check_backward(got, ins, dt, grow=D.joins(size[1]))


@pytest.mark.parametrize("Dk", [64, 128, 256])
def test_lengths_end_in_segments(Dk):
    """Padded sequences of slow decays that end at the segments' borders, inside and before the last of them."""
    S, L = 1600, [1600, 0, 300, 641, 1279, 1280]
    note(f"precision of padded segments Dk={Dk}")
    ins = D.inputs(len(L), S, 1, 1, Dk, 24, "f32", Dk, 1e-4)
    d = device(ins, "f32")
    lengths = torch.tensor(L, dtype=torch.int32, device="cuda")
    o, M = hc.hc_gated_delta(*d[:6], lengths=lengths)
    got = hc.hc_gated_delta_backward(*d[:5], d[6], d[5], d[7], lengths=lengths)
    torch.cuda.synchronize()
    check_forward(o, M, ins, "f32", L, grow=D.joins(S))
    check_backward(got, ins, "f32", L, grow=D.joins(S))
