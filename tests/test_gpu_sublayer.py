"""The norm, the gated scan, the balance loss and the router's backward on the GPU
against their float64 forms (oracle/sublayer_ops.py).

Tolerances, with u = 2^-24 the float32 rounding and p the rounding of the stored
type (0 for float32, 2^-8 for bfloat16), all relative to the magnitudes named:
  norm: a sum of squares is at most 32 terms of one thread, 6 steps over a wave and
    16 over a workgroup (54 u, halved by the root), the residual's sum, root, quotient
    and two products 6 u: 40 u in all on |y|; a pre-read of n terms adds (n + 1) u on
    the magnitude before cancellation, sum_i |h_i x_i| rstd |w|.
  8 bits: the scale and the division 44 u more, then half a step of the code: 2^-4
    |y| or half the smallest code 2^-10 scale (e4m3), 0.5 scale (int8).
  scan: with K = |gate| + 12 roundings per token for the sigmoid and the step (the
    exponential's argument is rounded once: |gate| u), the bound follows the state's own
    recurrence, e_t = a_t e_{t-1} + 2 K u (a_t |h_{t-1}| + |u_t x_t|).
"""
import numpy as np
import pytest

from hc_testutil import have_gpu, note
from oracle import sublayer_ops as R

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc

U = 2.0 ** -24
P = {"f32": 0.0, "bf16": 2.0 ** -8}


def _dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[name]


def up(a, dt="f32"):
    """(device tensor, its float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(_dt(dt))
    return t, t.float().cpu().numpy().astype(np.float64)


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def within(name, got, ref, tol):
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    bad = err > tol
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} off, worst {np.max(err / np.maximum(tol, 1e-300)):.3g} bounds"


# -------------------------------------------------------------------- norm

WIDTHS = [1, 7, 8, 33, 128, 500, 1000, 1024, 2048, 2050, 4096, 4100, 7168, 8200, 16384]


def _check_y(name, y, scale, ref, mag, dt, quant, group, n=1):
    """y (and its codes) against ref [T, C]; mag: the magnitude before cancellation."""
    tol = 40 * U * np.abs(ref) + (n + 1) * U * mag + 1e-37
    if quant is None:
        within(name, down(y), ref, tol + P[dt] * np.abs(ref))
        return
    T, C = ref.shape
    sref = R.quant_scales(ref, quant, group)
    width = group or C
    smag = np.stack([tol[:, c:c + width].max(1) for c in range(0, C, width)], 1) / R.QMAX[quant]
    within(name + " scale", down(scale), sref, 4 * U * sref + smag)
    s = R.per_channel(down(scale), C, group)
    half = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) if quant == "e4m3" else 0.5 * s
    within(name + " codes", down(y) * s, ref, half * (1 + 2.0 ** -10) + tol + 48 * U * np.abs(ref))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_with_residual(C, dt):
    rng = np.random.default_rng(C)
    for T, quant, group in ((5, None, 0), (3, "e4m3", 0), (6, "e4m3", 128), (2, "e4m3", 32), (4, "i8", 64),
                            (1, "i8", 0)):
        note(f"hc_rms_norm T={T} C={C} {dt} {quant} group={group}")
        x, x64 = up(rng.normal(size=(T, C)), dt)
        r, r64 = up(4 * rng.normal(size=(T, C)), dt)
        w, w64 = up(1 + 0.3 * rng.normal(size=C))
        q = None if quant is None else _dt(quant)
        got = hc.hc_rms_norm(x, w, 1e-5, residual=r, quant=q, group=group)
        torch.cuda.synchronize()
        v = x64 + r64
        ref = R.rms_norm(v, w64, 1e-5)
        within("s", down(got["s"]), v, (P[dt] + U) * np.abs(v))
        mag = (np.abs(x64) + np.abs(r64)) * np.abs(ref / np.where(v == 0, 1, v))
        _check_y("y", got["y"], got.get("scale"), ref, mag, dt, quant, group)


@pytest.mark.parametrize("T", [1, 2, 5, 9000])
def test_norm_without_residual_or_weight(T):
    note(f"hc_rms_norm T={T}, no residual, no weight")
    rng = np.random.default_rng(T)
    x, x64 = up(rng.normal(size=(T, 96)), "bf16")
    got = hc.hc_rms_norm(x, eps=0.0)
    assert set(got) == {"y"}
    _check_y("y", got["y"], None, R.rms_norm(x64, None, 0.0), np.abs(x64) * 0, "bf16", None, 0)


@pytest.mark.parametrize("n,C", [(1, 64), (3, 100), (4, 4096), (4, 7168), (16, 520), (64, 36)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pre_norm(n, C, dt):
    rng = np.random.default_rng(n * C)
    for T, quant, group in ((7, None, 0), (3, "e4m3", 64), (1, "i8", 0)):
        note(f"hc_pre_norm T={T} n={n} C={C} {dt} {quant}")
        X, X64 = up(rng.normal(size=(T, n, C)), dt)
        h, h64 = up(rng.uniform(0, 1, size=(T, n)))
        w, w64 = up(1 + 0.3 * rng.normal(size=C))
        got = hc.hc_pre_norm(X, h, w, 1e-6, quant=None if quant is None else _dt(quant), group=group)
        torch.cuda.synchronize()
        v = (h64[:, :, None] * X64).sum(1)
        mag = (np.abs(h64[:, :, None]) * np.abs(X64)).sum(1)
        within("F_in", down(got["F_in"]), v, P[dt] * np.abs(v) + (n + 1) * U * mag)
        rstd = np.abs(w64) / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
        _check_y("y", got["y"], got.get("scale"), R.rms_norm(v, w64, 1e-6), mag * rstd, dt, quant, group, n)
        # the two-call path: hc_pre, then the norm of what it stored (one more rounding of v)
        if quant is None and n <= 16:  # hc_pre takes up to 16 streams
            two = hc.hc_rms_norm(hc.hc_pre(X, h), w, 1e-6)["y"]
            within("two calls", down(two), down(got["y"]), (3 * P[dt] + 100 * U) * np.abs(down(two)) + 4 * n * U * mag * rstd)
            assert "F_in" not in hc.hc_pre_norm(X, h, w, want_F_in=False)


def test_norm_zero_rows_nan_and_infinity():
    note("hc_rms_norm zero, NaN and infinite rows")
    x = torch.randn(6, 300, device="cuda")
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    x[4] = 1e-30
    clean = hc.hc_rms_norm(x[5:].contiguous(), quant=_dt("e4m3"))
    for eps in (0.0, 1e-6):
        y = hc.hc_rms_norm(x, eps=eps)["y"]
        assert not y[1].any() and y[2].isnan().all() and y[3, 9].isnan() and not y[3, :9].any()
        got = hc.hc_rms_norm(x, eps=eps, quant=_dt("e4m3"))
        assert float(got["scale"][1]) == 1.0 and not got["y"][1].float().any()
        assert got["scale"][2].isnan() and got["y"][2].float().isnan().all()
        if eps:
            assert torch.equal(got["y"][5].float(), clean["y"][0].float())
    # groups keep a NaN to themselves
    x[2, 7] = 0.5
    w = torch.ones(300, device="cuda")
    w[70] = float("nan")
    got = hc.hc_rms_norm(x, w, quant=_dt("i8"), group=64)
    assert got["scale"][0].isnan().tolist() == [False, True, False, False, False]


def test_norm_in_place_residual_and_given_outputs():
    note("hc_rms_norm in place on the residual")
    x = torch.randn(9, 260, device="cuda").bfloat16()
    r = torch.randn(9, 260, device="cuda").bfloat16()
    want = hc.hc_rms_norm(x, residual=r, quant=_dt("e4m3"), group=32)
    y = torch.zeros(9, 260, dtype=_dt("e4m3"), device="cuda")
    sc = torch.zeros(9, 9, device="cuda")
    got = hc.hc_rms_norm(x, residual=r, s_out=r, quant=_dt("e4m3"), group=32, out=(y, sc))
    assert got["s"] is r and torch.equal(r, want["s"]) and torch.equal(y.view(torch.uint8), want["y"].view(torch.uint8))
    assert torch.equal(sc, want["scale"])


def test_norm_without_rows():
    note("hc_rms_norm, hc_pre_norm and the backward with T = 0")
    e = torch.empty(0, 64, device="cuda")
    r = hc.hc_rms_norm(e, torch.ones(64, device="cuda"), residual=e, quant=_dt("e4m3"), group=32)
    assert r["y"].shape == (0, 64) and r["s"].shape == (0, 64) and r["scale"].shape == (0, 2)
    assert hc.hc_pre_norm(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 4, device="cuda"))["y"].shape == (0, 64)
    dx, dw = hc.hc_rms_norm_backward(e, None, e)
    assert dx.shape == (0, 64) and dw.shape == (64,) and not dw.any()


def test_norm_unaligned_arrays():
    note("hc_rms_norm on arrays one element off a 16-byte address")
    for dt in ("bf16", "f32"):
        big = torch.randn(2 * 520 + 9, device="cuda").to(_dt(dt))
        x = big[1:1 + 2 * 520].view(2, 520)
        assert x.data_ptr() % 16
        y = hc.hc_rms_norm(x)["y"]
        dx, dw = hc.hc_rms_norm_backward(x, None, y)
        ax, aw = hc.hc_rms_norm_backward(x.clone(), None, y)
        assert torch.equal(y, hc.hc_rms_norm(x.clone())["y"]) and torch.equal(dx, ax) and torch.equal(dw, aw)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_backward(C, dt):
    rng = np.random.default_rng(C + 1)
    for T, with_ds in ((1, False), (6, True), (1100 if C <= 1024 else 515, True)):
        note(f"hc_rms_norm_backward T={T} C={C} {dt}")
        v, v64 = up(2 * rng.normal(size=(T, C)), dt)
        dy, dy64 = up(rng.normal(size=(T, C)), dt)
        ds, ds64 = up(rng.normal(size=(T, C)), dt)
        w, w64 = up(1 + 0.3 * rng.normal(size=C))
        dx, dw = hc.hc_rms_norm_backward(v, w, dy, 1e-6, ds=ds if with_ds else None)
        torch.cuda.synchronize()
        rx, rw = R.rms_norm_backward(v64, w64, 1e-6, dy64, ds64 if with_ds else None)
        rstd = 1 / np.sqrt((v64 * v64).mean(1, keepdims=True) + 1e-6)
        wdy = np.abs(w64 * dy64)
        mag = rstd * (wdy + np.abs(v64) * rstd * (wdy * np.abs(v64) * rstd).mean(1, keepdims=True))
        # each sum 54 u, the statistics in it twice: 120 u on the magnitudes; ds and the store round once
        within("dx", down(dx), rx, 120 * U * mag + (P[dt] + U) * np.abs(rx) + U * np.abs(ds64))
        # dw: rows of one walk in order, then the walks: at most (T + 60) roundings of the magnitudes
        within("dw", down(dw), rw, (T + 60) * U * (np.abs(dy64 * v64) * rstd).sum(0) + 1e-37)
        if with_ds:
            got, _ = hc.hc_rms_norm_backward(v, w, dy, 1e-6, ds=ds, out=(ds, None), want_dweight=False)
            assert got is ds and torch.equal(ds, dx)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [8193, 9001, 12288, 16383])
def test_norm_backward_of_rows_with_two_pieces_a_thread(C, dt):
    """Above 8,192 channels the weight and its gradient lie in LDS; the bounds are test_norm_backward's."""
    test_norm_backward(C, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T, C", [(9001, 8), (9001, 200), (4099, 511), (4500, 1032)])
def test_norm_backward_of_many_rows(T, C, dt):
    """Several rows a wave or workgroup: dw adds rows, waves and workgroups, T terms in all, each sum in
    at most T + 60 roundings of the magnitudes."""
    rng = np.random.default_rng(T + C)
    v, v64 = up(2 * rng.normal(size=(T, C)), dt)
    dy, dy64 = up(rng.normal(size=(T, C)), dt)
    w, w64 = up(1 + 0.3 * rng.normal(size=C))
    _, dw = hc.hc_rms_norm_backward(v, w, dy, 1e-6)
    torch.cuda.synchronize()
    _, rw = R.rms_norm_backward(v64, w64, 1e-6, dy64, None)
    rstd = 1 / np.sqrt((v64 * v64).mean(1, keepdims=True) + 1e-6)
    within("dw", down(dw), rw, (T + 60) * U * (np.abs(dy64 * v64) * rstd).sum(0) + 1e-37)


# --------------------------------------------------------------------- scan


def _scan_bound(a, b, K, init):
    """e_t of the recurrence s_t = a_t s_{t-1} + b_t (|b| given) over axis 1."""
    m, e = np.abs(init), np.zeros_like(init)
    es = np.zeros_like(a)
    for t in range(a.shape[1]):
        m = a[:, t] * m + np.abs(b[:, t])
        e = a[:, t] * e + 2 * K[:, t] * U * m
        es[:, t] = e
    return es


SCANS = [(1, 1, 1), (3, 1, 4096), (2, 2, 5), (1, 63, 64), (1, 64, 8), (2, 65, 66), (5, 129, 36), (1, 1021, 100),
         (2, 700, 260), (1, 5000, 12), (64, 3, 7)]


@pytest.mark.parametrize("B,S,C", SCANS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tied", [True, False])
def test_scan_forward_and_backward(B, S, C, dt, tied):
    note(f"hc_gated_scan B={B} S={S} C={C} {dt} tied={tied}")
    rng = np.random.default_rng(B * S + C)
    x, x64 = up(rng.normal(size=(B, S, C)), dt)
    g, g64 = up(rng.uniform(-2, 7, size=C) + rng.normal(size=(B, S, C)), dt)
    h0, h064 = up(rng.normal(size=(B, C)))
    dl, dl64 = up(rng.normal(size=(B, C)))
    dy, dy64 = up(rng.normal(size=(B, S, C)), dt)
    K = np.abs(g64) + 12
    a, u = R.sigmoid(g64), R.sigmoid(-g64) if tied else np.ones_like(g64)
    for L in (None, rng.integers(0, S + 1, size=B)):
        lengths = None if L is None else torch.from_numpy(L.astype(np.int32)).cuda()
        live = np.ones((B, S, 1), bool) if L is None else np.arange(S)[None, :, None] < L[:, None, None]
        y0, y064 = up(rng.normal(size=(B, S, C)), dt)
        y, last = hc.hc_gated_scan(x, g, h0, lengths=lengths, tied=tied, out=(y0.clone(), None))
        torch.cuda.synchronize()
        ry, rl = R.gated_scan(x64, g64, h064, L, tied, y064)
        al, bl = np.where(live, a, 1.0), np.where(live, u * x64, 0.0)
        e = _scan_bound(al, bl, np.where(live, K, 0.0), h064)
        got = down(y)
        assert np.array_equal(got[~live[:, :, 0]], y064[~live[:, :, 0]]), "rows behind the length changed"
        within("y", got, ry, np.where(live, e + P[dt] * (np.abs(ry) + e), 0))
        within("h_last", down(last), rl, e[:, -1] + 1e-30)

        y64 = down(y)
        dx, dg, d0 = hc.hc_gated_scan_backward(x, g, y, dy, h0, dl, lengths=lengths, tied=tied)
        torch.cuda.synchronize()
        rx, rg, r0 = R.gated_scan_backward(x64, g64, y64, dy64, h064, dl64, L, tied)
        # the reverse walk s <- a (dy + s): its bound at the step that enters token t
        back = lambda v: v[:, ::-1]  # noqa: E731
        eb = back(_scan_bound(back(al), back(np.where(live, a * np.abs(dy64), 0)), back(np.where(live, K, 0)), dl64))
        into = np.concatenate([eb[:, 1:], np.zeros((B, 1, C))], 1)  # error of R_t
        edh = into + 2 * U * (np.abs(dy64) + np.abs(rx / u))
        within("dx", down(dx), rx, np.where(live, u * edh + 2 * K * U * np.abs(rx) + P[dt] * np.abs(rx) * 1.01, 0))
        prev = np.concatenate([h064[:, None], y64[:, :-1]], 1)
        mag = np.abs(prev) + (np.abs(x64) if tied else 0)
        dh = np.abs(rx / u)
        tol = a * R.sigmoid(-g64) * mag * (edh + 6 * K * U * dh)
        within("dgate", down(dg), rg, np.where(live, tol + P[dt] * (np.abs(rg) + tol), 0))
        within("dh0", down(d0), r0, eb[:, 0] + 1e-30)


def test_scan_without_states_and_empty():
    note("hc_gated_scan without h0 and dh_last, S = 0 and B = 0")
    x, g = torch.randn(2, 130, 12, device="cuda"), torch.randn(2, 130, 12, device="cuda")
    z = torch.zeros(2, 12, device="cuda")
    y, last = hc.hc_gated_scan(x, g)
    y2, last2 = hc.hc_gated_scan(x, g, z)
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(y[:, -1], last)
    assert hc.hc_gated_scan(x, g, want_state=False)[1] is None
    a = hc.hc_gated_scan_backward(x, g, y, x)
    b = hc.hc_gated_scan_backward(x, g, y, x, z, z)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    h0 = torch.randn(2, 12, device="cuda")
    y, last = hc.hc_gated_scan(x[:, :0].contiguous(), g[:, :0].contiguous(), h0)
    assert y.shape == (2, 0, 12) and torch.equal(last, h0)
    e = x[:, :0].contiguous()
    assert torch.equal(hc.hc_gated_scan_backward(e, e, e, e, None, h0)[2], h0)
    y, last = hc.hc_gated_scan(x[:0].contiguous(), g[:0].contiguous())
    assert y.shape == (0, 130, 12)


def test_scan_goes_on_from_its_state():
    note("hc_gated_scan in pieces, the state in place")
    x, g = torch.randn(3, 300, 40, device="cuda").bfloat16(), 3 + torch.randn(3, 300, 40, device="cuda").bfloat16()
    h = torch.randn(3, 40, device="cuda")
    y, last = hc.hc_gated_scan(x, g, h)
    parts = []
    state = h.clone()
    for t0, t1 in ((0, 1), (1, 200), (200, 264), (264, 300)):
        yp, state2 = hc.hc_gated_scan(x[:, t0:t1].contiguous(), g[:, t0:t1].contiguous(), state, out=(None, state))
        assert state2 is state
        parts.append(yp)
    # each piece's state carries the float32 roundings of its own order
    assert torch.allclose(torch.cat(parts, 1).float(), y.float(), rtol=2.0 ** -7, atol=1e-5)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-5)


def test_scan_padding_may_hold_anything():
    note("hc_gated_scan with NaN behind the lengths")
    B, S, C = 3, 150, 20
    x, g, dy = (torch.randn(B, S, C, device="cuda") for _ in range(3))
    L = torch.tensor([150, 70, 0], dtype=torch.int32, device="cuda")
    y, last = hc.hc_gated_scan(x, g, lengths=L, out=(torch.zeros(B, S, C, device="cuda"), None))
    grads = hc.hc_gated_scan_backward(x, g, y, dy, lengths=L)
    dead = torch.arange(S, device="cuda")[None] >= L[:, None]
    x2, g2, dy2, yn = x.clone(), g.clone(), dy.clone(), y.clone()
    for t in (x2, g2, dy2, yn):
        t[dead] = float("nan")
    y2, last2 = hc.hc_gated_scan(x2, g2, lengths=L, out=(torch.zeros(B, S, C, device="cuda"), None))
    assert torch.equal(y, y2) and torch.equal(last, last2)
    for p, q in zip(grads, hc.hc_gated_scan_backward(x2, g2, yn, dy2, lengths=L)):
        assert torch.equal(p, q)
    # lengths out of range are taken as 0 and S
    L2 = torch.tensor([1 << 30, 70, -5], dtype=torch.int32, device="cuda")
    assert torch.equal(hc.hc_gated_scan(x, g, lengths=L2, out=(torch.zeros(B, S, C, device="cuda"), None))[0], y)


@pytest.mark.parametrize("where", ["x", "gate", "h0"])
def test_scan_nan_goes_on_in_its_channel(where):
    note(f"hc_gated_scan with a NaN of all ones in {where}")
    S, C = 2000, 300
    x, g = torch.randn(2, S, C, device="cuda"), torch.randn(2, S, C, device="cuda")
    h0 = torch.randn(2, C, device="cuda")
    y0, l0 = hc.hc_gated_scan(x, g, h0)
    ones = torch.full((1,), -1, dtype=torch.int32, device="cuda").view(torch.float32)
    t = 0 if where == "h0" else 150
    {"x": x, "gate": g, "h0": h0[:, None]}[where][1, t, 37] = ones[0]
    y, last = hc.hc_gated_scan(x, g, h0)
    torch.cuda.synchronize()
    assert y[1, t:, 37].isnan().all() and last[1, 37].isnan()
    y[1, t:, 37] = y0[1, t:, 37]
    last[1, 37] = l0[1, 37]
    assert torch.equal(y, y0) and torch.equal(last, l0)


def test_scan_gates_at_the_ends_of_their_range():
    note("hc_gated_scan with gates of -inf, +inf and the type's extremes")
    for dt in ("f32", "bf16"):
        x = torch.randn(1, 5, 8, device="cuda").to(_dt(dt))
        g = torch.zeros(1, 5, 8, device="cuda").to(_dt(dt))
        g[0, 1] = float("-inf")
        g[0, 2] = float("inf")
        g[0, 3] = torch.finfo(_dt(dt)).min
        g[0, 4] = torch.finfo(_dt(dt)).max
        h0 = torch.randn(1, 8, device="cuda")
        y, last = hc.hc_gated_scan(x, g, h0)
        assert torch.equal(y[0, 1], x[0, 1]) and torch.equal(y[0, 2], x[0, 1])
        assert torch.equal(y[0, 3], x[0, 3]) and torch.equal(y[0, 4], x[0, 3])
        dx, dg, d0 = hc.hc_gated_scan_backward(x, g, y, torch.ones_like(x), h0)
        assert torch.isfinite(dx).all() and torch.isfinite(dg).all() and not dg[0, 1:].any()


# ------------------------------------------------------------------- router


def _routing(rng, T, N, k, m):
    E = N - m
    score = rng.uniform(0.02, 0.98, size=(T, E)).astype(np.float32)
    idx = np.concatenate([np.tile(np.arange(m), (T, 1)), m + np.argsort(-score, 1)[:, :k - m]], 1)
    return score, np.sort(idx, 1).astype(np.int32)


@pytest.mark.parametrize("B,S,N,k,m", [(1, 1, 2, 2, 1), (1, 509, 8, 4, 1), (3, 257, 16, 4, 2), (40, 3, 12, 5, 1),
                                       (2, 600, 17, 6, 2), (1, 300, 64, 16, 1), (5, 1, 16, 3, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_loss(B, S, N, k, m, masked):
    note(f"xhc_balance_loss B={B} S={S} N={N} k={k} m={m} masked={masked}")
    rng = np.random.default_rng(B * S + N)
    T, E = B * S, N - m
    score, idx = _routing(rng, T, N, k, m)
    mask = rng.random(T) < 0.6 if masked else None
    if masked:
        mask[:S] = False  # a sequence without tokens
        score[~mask] = np.nan
        score[0] = np.inf
        idx[~mask] = 1 << 20
    ts, ti = torch.from_numpy(score).cuda(), torch.from_numpy(idx).cuda()
    tm = None if mask is None else torch.from_numpy(mask).cuda()
    got = hc.xhc_balance_loss(ts, ti, B, S, m=m, coef=0.01, mask=tm)
    dl = torch.full((1,), 3.0, device="cuda")
    ds = hc.xhc_balance_loss_backward(ts, got["count"], got["tokens"], k, B, S, coef=0.01, dloss=dl, mask=tm)
    torch.cuda.synchronize()
    ref = R.balance_loss(score, idx, B, S, N, m, 0.01, mask)
    rd = R.balance_loss_backward(score, ref["count"], ref["tokens"], k, B, S, N, m, 0.01, 3.0, mask)
    assert np.array_equal(got["count"].cpu().numpy(), ref["count"])
    assert np.array_equal(got["tokens"].cpu().numpy(), ref["tokens"])
    # a token's sum 6 u, its quotient 1 u, then at most 16 + 16 + S/256 + 4 ordered additions of positive terms
    tol = (44 + S / 256) * U
    within("mean_p", down(got["mean_p"]), ref["mean_p"], tol * ref["mean_p"] + 1e-37)
    within("loss", down(got["loss"]), np.array(ref["loss"]), (tol + (B + 16) * U) * abs(ref["loss"]) + 1e-37)
    # f and the weighted mean of f: 16 u each on the larger of the two, over the sum of the scores
    n = np.maximum(ref["tokens"], 1)[:, None]
    f = ref["count"][:, m:] * E / ((k - m) * n)
    live = np.ones(T, bool) if mask is None else mask
    total = np.where(live[:, None], score, 1.0).astype(np.float64).sum(1, keepdims=True)
    fmax = np.repeat(f.max(1), S)[:, None] if S else f
    within("dscore", down(ds), rd, 32 * U * 0.03 / (B * np.repeat(n, S, 0)) * fmax / total + 1e-37)
    assert not down(ds)[~live].any()
    if not masked:
        one = hc.xhc_balance_loss_backward(ts, got["count"], got["tokens"], k, B, S, coef=0.03)
        within("dloss", down(one), down(ds), 4 * U * np.abs(down(ds)) + 1e-37)


def test_balance_loss_empty_and_zero_scores():
    note("xhc_balance_loss with no tokens, and with scores that are all zero")
    e = torch.empty(0, 6, device="cuda")
    r = hc.xhc_balance_loss(e, torch.empty(0, 4, dtype=torch.int32, device="cuda"), 2, 0, m=2)
    assert float(r["loss"]) == 0 and not r["count"].any() and not r["tokens"].any() and not r["mean_p"].any()
    assert hc.xhc_balance_loss_backward(e, r["count"], r["tokens"], 4, 2, 0).shape == (0, 6)
    r = hc.xhc_balance_loss(e, torch.empty(0, 4, dtype=torch.int32, device="cuda"), 0, 5, m=2)
    assert float(r["loss"]) == 0
    z = torch.zeros(3, 6, device="cuda")
    idx = torch.tensor([[0, 1, 2, 3]] * 3, dtype=torch.int32, device="cuda")
    r = hc.xhc_balance_loss(z, idx, 1, 3, m=2)
    assert float(r["loss"]) == 0 and r["count"][0].tolist() == [3, 3, 3, 3, 0, 0, 0, 0]
    assert not hc.xhc_balance_loss_backward(z, r["count"], r["tokens"], 4, 1, 3).any()


@pytest.mark.parametrize("T,N,m,C", [(1, 2, 1, 32), (33, 4, 3, 64), (100, 8, 2, 96), (257, 16, 2, 512), (70, 16, 1, 1024),
                                     (40, 13, 1, 160), (5, 16, 4, 4096), (1100, 6, 2, 32)])
def test_router_backward(T, N, m, C):
    note(f"xhc_router_backward T={T} N={N} m={m} C={C}")
    rng = np.random.default_rng(T + N)
    E = N - m
    X, X64 = up(rng.normal(size=(T, N, C)), "bf16")
    dX, dX64 = up(0.05 * rng.normal(size=(T, N, C)), "bf16")
    w, w64 = up(rng.normal(size=(N * C, E)) * 2 / np.sqrt(N * C))
    x = X64.reshape(T, -1)
    rr = np.sqrt((x * x).mean(1, keepdims=True))
    score, s64 = up(R.sigmoid((x @ w64) / rr))
    ds, ds64 = up(rng.normal(size=(T, E)))
    if T > 4:
        ds[2] = 0  # takes no part, whatever its row holds
        ds64[2] = 0
        X[2] = float("nan")
        X64[2] = np.nan
        score[2] = float("nan")
        s64[2] = np.nan
        X[3] = 0  # the all-zero state passes nothing
        X64[3] = 0
    out, dw = hc.xhc_router_backward(X, w, score, ds, dX, out=torch.full_like(dX, float("nan")))
    torch.cuda.synchronize()
    ref, rdw = R.router_backward(X64, w64, s64, ds64, dX64)
    live = (ds64 != 0).any(1) & np.array([np.any(v != 0) for v in X64])
    xl, sl, dl = x[live], s64[live], ds64[live]
    rl = np.sqrt((xl * xl).mean(1, keepdims=True))
    dz = np.abs(dl * sl * (1 - sl))
    z = np.abs(np.log(sl) - np.log1p(-sl))
    # r: at most NC / 256 + 10 ordered additions, halved by the root; the logit's logarithms 4 u on (1 + |z|) terms
    kr = (N * C / 256 + 10) / 2 + 8
    mag = np.zeros((T, N * C))
    mag[live] = (dz / rl) @ np.abs(w64).T * (kr + E + 4) + np.abs(xl) / (rl * rl * N * C) * (
        (dz * (z + 1)).sum(1, keepdims=True) * (2 * kr + 16))
    # dX's product takes P and w in two bfloat16 parts each: what is left of either is at most 2^-8 of 2^-8 of it
    split = np.zeros((T, N * C))
    split[live] = 2 * 2.0 ** -16 * ((dz / rl) @ np.abs(w64).T)
    tol = U * (mag.reshape(T, N, C) + 4 * np.abs(dX64)) + split.reshape(T, N, C)
    within("dX", down(out), ref, tol + P["bf16"] * (np.abs(ref) + tol))
    wmag = np.abs(xl).T @ (dz / rl)
    within("dw", down(dw), rdw, (kr + 4 + T) * U * wmag + 1e-37)
    same, dw2 = hc.xhc_router_backward(X, w, score, ds, dX)
    assert same is dX and torch.equal(dX, out) and torch.equal(dw, dw2)


def test_router_backward_without_tokens():
    note("xhc_router_backward T=0")
    X = torch.empty(0, 4, 32, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 2, device="cuda")
    _, dw = hc.xhc_router_backward(X, torch.ones(128, 2, device="cuda"), e, e, X.clone())
    assert dw.shape == (128, 2) and not dw.any()
