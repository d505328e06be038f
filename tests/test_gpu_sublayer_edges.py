"""The norm, the scan and the router's backward at the edges of what their definitions allow:
padded batches whose output the call allocates, rows whose squares leave float32's range,
infinite states, workspaces with anything in them, and the smallest and largest states."""
import numpy as np
import pytest

from hc_testutil import have_gpu, note
from oracle import sublayer_ops as R
from test_gpu_sublayer import P, U, _check_y, _dt, down, up, within

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc


# ------------------------------------------------- padding of an allocated y


def _dirty(shape, dtype):
    """Leaves NaN in the allocator's free memory of this size."""
    junk = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("S", [1, 20, 100, 600])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_padding_of_an_allocated_output_is_zero(S, dt):
    note(f"hc_gated_scan with lengths and no out, S={S} {dt}")
    B, C = 4, 512
    x, g = (torch.randn(B, S, C, device="cuda").to(_dt(dt)) for _ in range(2))
    L = torch.tensor([S, S // 2, 0, -3], dtype=torch.int32, device="cuda")
    want, last = hc.hc_gated_scan(x, g, lengths=L, out=(torch.zeros_like(x), None))
    for out in (None, (None, None), (None, torch.empty(B, C, device="cuda"))):
        _dirty((B, S, C), x.dtype)
        y, l2 = hc.hc_gated_scan(x, g, lengths=L, out=out)
        assert torch.equal(y, want) and torch.equal(l2, last)
    # what a following norm makes of it: padded rows with dy = 0 add nothing to the weight's gradient
    _dirty((B, S, C), x.dtype)
    y, _ = hc.hc_gated_scan(x, g, lengths=L)
    dy = torch.ones_like(y)
    dy[torch.arange(S, device="cuda")[None] >= L[:, None]] = 0
    dx, dw = hc.hc_rms_norm_backward(y.view(B * S, C), None, dy.view(B * S, C))
    assert torch.isfinite(dw).all() and torch.isfinite(dx).all()


def test_scan_padding_of_an_allocated_output_in_a_graph():
    note("hc_gated_scan with lengths and no out, captured and replayed")
    B, S, C = 3, 200, 256
    x, g = (torch.randn(B, S, C, device="cuda").bfloat16() for _ in range(2))
    L = torch.tensor([S, 7, 0], dtype=torch.int32, device="cuda")
    hc.hc_gated_scan(x, g, lengths=L)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = hc.hc_gated_scan(x, g, lengths=L)
    for lens in ([S, 7, 0], [3, S, 150], [0, 0, 0]):
        L.copy_(torch.tensor(lens, dtype=torch.int32))
        y.fill_(float("nan"))
        graph.replay()
        want, wl = hc.hc_gated_scan(x, g, lengths=L, out=(torch.zeros_like(x), None))
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(last, wl)


# ------------------------------------- rows whose squares leave float32's range

# magnitudes of rows: squares over and under float32's range, its ends, and one in the middle
SIZES = [2e19, 1e20, 1e30, 3e37, 1.0, 3e-22, 1e-23, 1e-30, 1e-38, 1e-41]
DENORMAL = 2.0 ** -149


def _rows(rng, C, dt):
    """Rows of the magnitudes above, and mixed ones: one channel far beyond the others."""
    v = rng.normal(size=(len(SIZES) + 4, C))
    v[:len(SIZES)] *= np.array(SIZES)[:, None]
    v[-4, 0] = 1e30
    v[-3] *= 1e-30
    v[-3, C - 1] = 1e-20
    v[-2] *= 1e25
    v[-2, C // 2] = -3e38
    v[-1] = 0
    return up(v, dt)


@pytest.mark.parametrize("C", [1, 7, 128, 500, 1000, 2050, 4096, 9001])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_of_rows_beyond_the_squares_range(C, dt):
    """Scaling a row by a power of two is exact: the bounds are those of rows in range, and one step
    of the smallest stored numbers (2^-133 bfloat16, 2^-149 float32: half of it for each of two roundings)."""
    rng = np.random.default_rng(C)
    x, x64 = _rows(rng, C, dt)
    w, w64 = up(1 + 0.3 * rng.normal(size=C))
    for eps in (0.0, 1e-6, 1e-32, 1e-41, 1e30):
        e64 = float(np.float32(eps))
        ref = R.rms_norm(x64, w64, e64)
        note(f"hc_rms_norm of large and small rows C={C} {dt} eps={eps}")
        y = hc.hc_rms_norm(x, w, eps)["y"]
        tol = (40 * U + P[dt]) * np.abs(ref) + 2.0 ** (-133 if dt == "bf16" else -149)
        within(f"y eps={eps}", down(y), ref, tol)
        for quant, group in (("e4m3", 0), ("i8", 64)):
            got = hc.hc_rms_norm(x, w, eps, quant=_dt(quant), group=group)
            keep = np.abs(ref).max(1) > 1e-30  # smaller rows take the scale 1, or one at its border
            _check_y(f"{quant} eps={eps}", got["y"][torch.from_numpy(keep).cuda()],
                     got["scale"][torch.from_numpy(keep).cuda()], ref[keep], 0 * ref[keep], dt, quant, group)


@pytest.mark.parametrize("C", [36, 520, 4096])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_residual_and_pre_norm_beyond_the_squares_range(C, dt):
    rng = np.random.default_rng(C + 2)
    x, x64 = _rows(rng, C, dt)
    T = x.shape[0]
    note(f"hc_rms_norm with residual and hc_pre_norm of large and small rows C={C} {dt}")
    # x + x/2: exact in float64, no cancellation
    r = x / 2
    v = x64 + r.double().cpu().numpy()
    for eps in (0.0, 1e-6):
        e64 = float(np.float32(eps))
        big = np.abs(v) > 3.3e38  # sums past float32's range are infinite by definition
        assert not big[:-4].any()
        ok = ~big.any(1)
        got = hc.hc_rms_norm(x, None, eps, residual=r)
        ref = R.rms_norm(v, None, e64)
        tol = (44 * U + P[dt]) * np.abs(ref) + 2.0 ** (-133 if dt == "bf16" else -149)
        within("y", down(got["y"])[ok], ref[ok], tol[ok])
        within("s", down(got["s"])[ok], v[ok], ((P[dt] + U) * np.abs(v) + 2.0 ** -134)[ok])
        X = torch.stack([x, r], 1)
        h = torch.ones(T, 2, device="cuda")
        pre = hc.hc_pre_norm(X, h, None, eps)
        within("pre y", down(pre["y"])[ok], ref[ok], tol[ok])


@pytest.mark.parametrize("C", [1, 7, 128, 500, 1000, 4096, 8200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_backward_of_rows_beyond_the_squares_range(C, dt):
    """test_norm_backward's bounds on the magnitudes, and one step of the smallest stored numbers. dy is
    small where the row is, so that dx stays in range."""
    rng = np.random.default_rng(C + 1)
    v, v64 = _rows(rng, C, dt)
    T = v.shape[0]
    g = rng.normal(size=(T, C))
    g[np.abs(v64).max(1) < 1e-25] *= 1e-12
    dy, dy64 = up(g, dt)
    w, w64 = up(1 + 0.3 * rng.normal(size=C))
    for eps in (0.0, 1e-6, 1e-32):
        note(f"hc_rms_norm_backward of large and small rows C={C} {dt} eps={eps}")
        e64 = float(np.float32(eps))
        dx, dw = hc.hc_rms_norm_backward(v, w, dy, eps)
        torch.cuda.synchronize()
        rx, rw = R.rms_norm_backward(v64, w64, e64, dy64)
        ms = (v64 * v64).mean(1, keepdims=True) + e64
        rstd = np.where(ms > 0, 1 / np.sqrt(np.where(ms > 0, ms, 1)), 0)
        wdy = np.abs(w64 * dy64)
        vh = np.abs(v64) * rstd
        mag = rstd * (wdy + vh * (wdy * vh).mean(1, keepdims=True))
        within(f"dx eps={eps}", down(dx), rx,
               120 * U * mag + (P[dt] + U) * np.abs(rx) + 2.0 ** (-133 if dt == "bf16" else -149))
        within(f"dw eps={eps}", down(dw), rw, (T + 60) * U * (np.abs(dy64) * vh).sum(0) + 1e-37)


# ------------------------------------------------------------ infinite states


@pytest.mark.parametrize("S", [5, 40, 129, 300, 1100, 2500])
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_keeps_an_infinite_state(S, tied, dt):
    """Every a is above 0, so an infinite state stays infinite whatever the sequence's length, until
    an infinity of the other sign meets it; the other channels give what they give without it."""
    note(f"hc_gated_scan with infinities S={S} tied={tied} {dt}")
    B, C = 2, 130
    gen = torch.Generator(device="cuda").manual_seed(S)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, g = rn(B, S, C).to(_dt(dt)), (rn(B, S, C) - 2).to(_dt(dt))  # a of about 0.12: products underflow
    h0, dy, dl = rn(B, C), rn(B, S, C).to(_dt(dt)), rn(B, C)
    y0, l0 = hc.hc_gated_scan(x, g, h0, tied=tied)
    x2, h2 = x.clone(), h0.clone()
    inf = float("inf")
    h2[0, 3], h2[1, 70], h2[0, 129] = inf, -inf, inf
    x2[0, 4, 9], x2[1, S // 2, 64], x2[0, S - 1, 65] = -inf, inf, inf
    x2[0, S // 2, 129] = -inf  # meets the other infinity: NaN from there on
    y, last = hc.hc_gated_scan(x2, g, h2, tied=tied)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ry, rl = R.gated_scan(down(x2), down(g), down(h2), None, tied)
    odd = ~np.isfinite(ry)
    got, gl = down(y), down(last)
    assert np.array_equal(np.isnan(got), np.isnan(ry)) and np.array_equal(got[np.isinf(ry)], ry[np.isinf(ry)])
    assert np.array_equal(np.isnan(gl), np.isnan(rl)) and np.array_equal(gl[np.isinf(rl)], rl[np.isinf(rl)])
    assert np.array_equal(got[~odd], down(y0)[~odd]) and np.array_equal(gl[np.isfinite(rl)], down(l0)[np.isfinite(rl)])

    # backward: infinite gradients pass on to the earlier tokens
    dx0, dg0, d0 = hc.hc_gated_scan_backward(x, g, y0, dy, h0, dl, tied=tied)
    dy2, dl2 = dy.clone(), dl.clone()
    dl2[0, 3], dl2[1, 70], dl2[0, 129] = inf, -inf, inf
    dy2[0, S - 2, 9], dy2[1, S // 2, 64], dy2[0, 0, 65] = -inf, inf, inf
    dx, dg, dh = hc.hc_gated_scan_backward(x, g, y0, dy2, h0, dl2, tied=tied)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ref = R.gated_scan_backward(down(x), down(g), down(y0), down(dy2), down(h0), down(dl2), None, tied)
    for name, t, clean, r in zip(("dx", "dgate", "dh0"), (dx, dg, dh), (dx0, dg0, d0), ref):
        t, clean = down(t), down(clean)
        assert np.array_equal(np.isnan(t), np.isnan(r)), name
        assert np.array_equal(t[np.isinf(r)], r[np.isinf(r)]), name
        assert np.array_equal(t[np.isfinite(r)], clean[np.isfinite(r)]), name


def test_scan_map_of_closed_gates_forgets():
    """A gate that closes fully (a = 0) resets the state: nothing of what was before is left, in any
    form of the scan."""
    note("hc_gated_scan with closed gates after a large state")
    for S in (20, 300, 1500):
        x = torch.zeros(1, S, 64, device="cuda")
        g = torch.zeros(1, S, 64, device="cuda")
        g[0, S // 3] = float("-inf")
        h0 = torch.full((1, 64), 3e38, device="cuda")
        y, last = hc.hc_gated_scan(x, g, h0)
        assert not y[0, S // 3:].any() and not last.any() and bool((y[0, 0] > 1e38).all())


def test_scan_workspace_with_anything_in_it_used_by_one_call_after_another():
    """One workspace for calls of other sizes, in order on one stream, eager and captured."""
    note("hc_gated_scan with a shared workspace that holds anything")
    gen = torch.Generator(device="cuda").manual_seed(31)
    cases = []
    for B, S, C in ((1, 3000, 130), (3, 300, 512), (2, 129, 64)):
        x, g = (torch.randn(B, S, C, device="cuda", generator=gen) for _ in range(2))
        cases.append((x, g, hc.hc_gated_scan(x, g)))
    n = max(hc.hc_gated_scan_workspace_bytes(*x.shape) for x, _, _ in cases)
    graphs = []
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for x, g, _ in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = hc.hc_gated_scan(x, g, workspace=ws)
        graphs.append((graph, out))
    for fill in (0, 255, 1, None):
        if fill is None:
            ws.random_(generator=gen)
        else:
            ws.fill_(fill)
        for (x, g, want), (graph, out) in zip(cases, graphs):
            y, last = hc.hc_gated_scan(x, g, workspace=ws)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[0]) and torch.equal(last, want[1])
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


# ------------------------------------------------ the router's range of states


@pytest.mark.parametrize("size", [1e-18, 1e-9, 1e6, 1e15])
def test_router_backward_over_its_range_of_states(size):
    """test_router_backward's bounds where r is at the ends of the stated range (dX = 0: the router's part alone)."""
    note(f"xhc_router_backward with states of size {size}")
    rng = np.random.default_rng(7)
    T, N, m, C = 70, 16, 2, 512
    E = N - m
    x = rng.normal(size=(T, N, C))
    x *= size / np.sqrt((x * x).mean((1, 2), keepdims=True))
    X, X64 = up(x * (1.01 if size < 1 else 0.99), "bf16")  # inside the range after rounding
    w, w64 = up(rng.normal(size=(N * C, E)) * 2 / np.sqrt(N * C))
    xf = X64.reshape(T, -1)
    r = np.sqrt((xf * xf).mean(1, keepdims=True))
    score, s64 = up(R.sigmoid((xf @ w64) / r))
    ds, ds64 = up(rng.normal(size=(T, E)))
    out, dw = hc.xhc_router_backward(X, w, score, ds, torch.zeros_like(X), out=torch.empty_like(X))
    torch.cuda.synchronize()
    ref, rdw = R.router_backward(X64, w64, s64, ds64, np.zeros_like(X64))
    dz = np.abs(ds64 * s64 * (1 - s64))
    z = np.abs(np.log(s64) - np.log1p(-s64))
    kr = (N * C / 256 + 10) / 2 + 8
    prod = (dz / r) @ np.abs(w64).T
    along = np.abs(xf) / (r * r * N * C) * ((dz * (z + 1)).sum(1, keepdims=True) * (2 * kr + 16))
    tol = (U * (prod * (kr + E + 4) + along) + 2 * 2.0 ** -16 * prod).reshape(T, N, C)
    within("dX", down(out), ref, tol + P["bf16"] * (np.abs(ref) + tol))
    within("dw", down(dw), rdw, (kr + 4 + T) * U * (np.abs(xf).T @ (dz / r)) + 1e-37)
