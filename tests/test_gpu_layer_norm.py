"""The layer norm and its backward on the GPU against their float64 forms (oracle/sublayer_ops.py).

Tolerances, with u = 2^-24 the float32 rounding and p the rounding of the stored type (0 for
float32, 2^-8 for bfloat16); a sum over a row's threads is at most 54 roundings (as for the
root-mean-square norm):
  deviation d = v - mean: one rounding of its own, the mean's remainder (54 u of mean|d|, and
    the deviations' roundings in it) and one more: 60 u (|d| + mean|d|);
  1 / sqrt(var): 54 u and the deviations' 120 u halved, root and quotient: 120 u; three more
    roundings for weight and bias. In all 200 u |w| rstd (|d| + mean|d|) + 2 u |b|;
  a residual's sum or a pre-read of n terms adds (n + 1) u on the magnitudes before
    cancellation and on their mean, over the standard deviation.
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
WIDTHS = [1, 7, 8, 33, 128, 500, 512, 520, 1100, 2048, 2050, 4096, 7168, 8200, 16384]


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


def _mean(a):
    return a.mean(1, keepdims=True)


def _moments(v, eps):
    d = v - _mean(v)
    return d, 1 / np.sqrt(_mean(d * d) + eps)


def _tol(v, eps, w, b, mag, n):
    """Bound on y before its last rounding; mag: the magnitudes that make up v."""
    d, rstd = _moments(v, eps)
    return np.abs(w) * rstd * (200 * U * (np.abs(d) + _mean(np.abs(d))) + (n + 1) * U * (mag + _mean(mag))) + \
        2 * U * np.abs(b) + 1e-37


def _check_y(y, scale, ref, tol, dt, quant, group):
    if quant is None:
        within("y", down(y), ref, tol + P[dt] * (np.abs(ref) + tol))
        return
    T, C = ref.shape
    sref = R.quant_scales(ref, quant, group)
    width = group or C
    smag = np.stack([tol[:, c:c + width].max(1) for c in range(0, C, width)], 1) / R.QMAX[quant]
    within("scale", down(scale), sref, 4 * U * sref + smag)
    s = R.per_channel(down(scale), C, group)
    half = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) if quant == "e4m3" else 0.5 * s
    # the code is that of a value off by tol, over a scale with 4 roundings of its own
    within("codes", down(y) * s, ref, half * (1 + 2.0 ** -10) + 1.1 * tol + 8 * U * np.abs(ref))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_with_residual(C, dt):
    rng = np.random.default_rng(C)
    for T, quant, group in ((5, None, 0), (3, "e4m3", 0), (6, "e4m3", 128), (2, "e4m3", 32), (4, "i8", 64),
                            (1, "i8", 0)):
        note(f"hc_layer_norm T={T} C={C} {dt} {quant} group={group}")
        x, x64 = up(rng.normal(size=(T, C)), dt)
        r, r64 = up(4 * rng.normal(size=(T, C)) + 2, dt)
        w, w64 = up(1 + 0.3 * rng.normal(size=C))
        b, b64 = up(0.3 * rng.normal(size=C))
        got = hc.hc_layer_norm(x, w, b, 1e-5, residual=r, quant=None if quant is None else _dt(quant), group=group)
        torch.cuda.synchronize()
        v = x64 + r64
        within("s", down(got["s"]), v, (P[dt] + U) * np.abs(v))
        _check_y(got["y"], got.get("scale"), R.layer_norm(v, w64, b64, 1e-5),
                 _tol(v, 1e-5, w64, b64, np.abs(x64) + np.abs(r64), 1), dt, quant, group)


@pytest.mark.parametrize("T", [1, 2, 5, 9000])
def test_without_residual_weight_or_bias(T):
    note(f"hc_layer_norm T={T}, no residual, weight or bias")
    x, x64 = up(np.random.default_rng(T).normal(size=(T, 96)), "bf16")
    got = hc.hc_layer_norm(x, eps=0.0)
    assert set(got) == {"y"}
    _check_y(got["y"], None, R.layer_norm(x64, None, None, 0.0), _tol(x64, 0.0, 1.0, 0.0, 0 * x64, 0), "bf16", None, 0)


@pytest.mark.parametrize("n,C", [(1, 64), (3, 100), (4, 4096), (4, 7168), (16, 520), (64, 36)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pre_read(n, C, dt):
    rng = np.random.default_rng(n * C)
    for T, quant, group in ((7, None, 0), (3, "e4m3", 64), (1, "i8", 0)):
        note(f"hc_pre_layer_norm T={T} n={n} C={C} {dt} {quant}")
        X, X64 = up(rng.normal(size=(T, n, C)), dt)
        h, h64 = up(rng.uniform(0, 1, size=(T, n)))
        w, w64 = up(1 + 0.3 * rng.normal(size=C))
        b, b64 = up(0.3 * rng.normal(size=C))
        got = hc.hc_pre_layer_norm(X, h, w, b, 1e-6, quant=None if quant is None else _dt(quant), group=group)
        torch.cuda.synchronize()
        v = (h64[:, :, None] * X64).sum(1)
        mag = (np.abs(h64[:, :, None]) * np.abs(X64)).sum(1)
        within("F_in", down(got["F_in"]), v, P[dt] * np.abs(v) + (n + 1) * U * mag)
        _check_y(got["y"], got.get("scale"), R.layer_norm(v, w64, b64, 1e-6), _tol(v, 1e-6, w64, b64, mag, n), dt,
                 quant, group)
    assert "F_in" not in hc.hc_pre_layer_norm(X, h, w, want_F_in=False)


@pytest.mark.parametrize("C", WIDTHS + [8193, 9001, 16383])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward(C, dt):
    rng = np.random.default_rng(C + 1)
    for T, with_ds in ((1, False), (6, True), (1100 if C <= 1100 else 515, True)):
        note(f"hc_layer_norm_backward T={T} C={C} {dt}")
        v, v64 = up(2 * rng.normal(size=(T, C)) + 1, dt)
        dy, dy64 = up(rng.normal(size=(T, C)), dt)
        ds, ds64 = up(rng.normal(size=(T, C)), dt)
        w, w64 = up(1 + 0.3 * rng.normal(size=C))
        dx, dw, db = hc.hc_layer_norm_backward(v, w, dy, 1e-5, ds=ds if with_ds else None)
        torch.cuda.synchronize()
        rx, rw, rb = R.layer_norm_backward(v64, w64, 1e-5, dy64, ds64 if with_ds else None)
        d, rstd = _moments(v64, 1e-5)
        n = rstd * (np.abs(d) + _mean(np.abs(d)))
        u = np.abs(w64 * dy64)
        mag = rstd * (u + _mean(u) + n * _mean(u * n))
        # n is off by 200 u of its bound, twice in the last term, the sums by 54 u each
        within("dx", down(dx), rx, 600 * U * mag + (P[dt] + U) * np.abs(rx) + U * np.abs(ds64) + 1e-37)
        within("dw", down(dw), rw, (T + 260) * U * (np.abs(dy64) * n).sum(0) + 1e-37)
        within("db", down(db), rb, (T + 60) * U * np.abs(dy64).sum(0) + 1e-37)
        if with_ds:
            got, none, none2 = hc.hc_layer_norm_backward(v, w, dy, 1e-5, ds=ds, out=(ds, None, None), want_dweight=False)
            assert got is ds and torch.equal(ds, dx) and none is None and none2 is None
    only = torch.empty(C, device="cuda")
    _, none, got = hc.hc_layer_norm_backward(v, w, dy, 1e-5, out=(None, None, only), want_dweight=False)
    assert none is None and got is only and torch.equal(only, db)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T, C", [(9001, 8), (9001, 200), (4099, 511), (4500, 1032)])
def test_backward_of_many_rows(T, C, dt):
    """Several rows a wave or workgroup; the bounds are test_backward's."""
    note(f"hc_layer_norm_backward T={T} C={C} {dt}")
    rng = np.random.default_rng(T + C)
    v, v64 = up(2 * rng.normal(size=(T, C)), dt)
    dy, dy64 = up(rng.normal(size=(T, C)), dt)
    _, dw, db = hc.hc_layer_norm_backward(v, None, dy, 1e-5)
    torch.cuda.synchronize()
    _, rw, rb = R.layer_norm_backward(v64, None, 1e-5, dy64)
    d, rstd = _moments(v64, 1e-5)
    within("dw", down(dw), rw, (T + 260) * U * (np.abs(dy64) * rstd * (np.abs(d) + _mean(np.abs(d)))).sum(0))
    within("db", down(db), rb, (T + 60) * U * np.abs(dy64).sum(0))


@pytest.mark.parametrize("C", [8, 300, 1000, 5000, 16384])
def test_rows_far_from_zero_and_of_equal_values(C):
    """Deviations of a few last bits around a large mean: d is exact there (Sterbenz), so the bound on y is
    that of any other row, with no term in the mean."""
    note(f"hc_layer_norm C={C}: rows far from zero")
    rng = np.random.default_rng(C)
    off = np.array([1e4, -3e6, 1.0, 1e30, -1e-25, 2e38, 7.0])[:, None]
    steps = rng.integers(-8, 9, size=(7, C)) * 2.0 ** -23
    steps[6] = 0
    x, x64 = up(off * (1 + steps))
    dy, dy64 = up(rng.normal(size=(7, C)))
    for eps in (0.0, 1e-6):
        y = hc.hc_layer_norm(x, eps=eps)["y"]
        dx, dw, db = hc.hc_layer_norm_backward(x, None, dy, eps)
        torch.cuda.synchronize()
        ref = R.layer_norm(x64, None, None, eps)
        d = x64 - _mean(x64)
        var = _mean(d * d) + eps
        rstd = np.where(var > 0, 1 / np.sqrt(np.where(var > 0, var, 1)), 0)
        n = rstd * (np.abs(d) + _mean(np.abs(d)))
        within("y", down(y), ref, 200 * U * n)
        assert not y[6].any()
        rx, rw, _ = R.layer_norm_backward(x64, None, eps, dy64)
        mag = rstd * (np.abs(dy64) + _mean(np.abs(dy64)) + n * _mean(np.abs(dy64) * n))
        within("dx", down(dx), rx, np.minimum(600 * U * mag, 1e38) + 1e-37)
        within("dw", down(dw), rw, 267 * U * (np.abs(dy64) * n).sum(0))


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-9, 1e9, 1e15, 1e20, 1e37])
def test_magnitudes_over_the_whole_range(size):
    """Scaling by a power of two is exact: the bounds are those of rows of size 1. dx is at most
    600 u mag off, or half a step of the smallest normal number's binade."""
    note(f"hc_layer_norm rows of {size}")
    rng = np.random.default_rng(3)
    for C in (100, 1100, 9000):
        x, x64 = up(size * (rng.normal(size=(4, C)) + 0.5))
        dy, dy64 = up(rng.normal(size=(4, C)))
        y = hc.hc_layer_norm(x, eps=0.0)["y"]
        dx, dw, _ = hc.hc_layer_norm_backward(x, None, dy, 0.0)
        torch.cuda.synchronize()
        d, rstd = _moments(x64, 0.0)
        n = rstd * (np.abs(d) + _mean(np.abs(d)))
        # values below the smallest normal number are read with what the type holds of them
        within("y", down(y), R.layer_norm(x64, None, None, 0.0), 200 * U * n)
        rx, rw, _ = R.layer_norm_backward(x64, None, 0.0, dy64)
        mag = rstd * (np.abs(dy64) + _mean(np.abs(dy64)) + n * _mean(np.abs(dy64) * n))
        big = mag * 4 > 3e38
        got, want = down(dx), rx
        within("dx", np.where(big, 0, got), np.where(big, 0, want), 600 * U * mag + 2.0 ** -149)
        within("dw", down(dw), rw, 264 * U * (np.abs(dy64) * n).sum(0))


def test_nan_and_infinity_stay_in_their_row():
    note("hc_layer_norm NaN and infinite rows")
    for C in (300, 1300):
        x = torch.randn(5, C, device="cuda")
        clean = hc.hc_layer_norm(x)["y"]
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        x[3] = float("-inf")
        y = hc.hc_layer_norm(x)["y"]
        assert y[1:4].isnan().all() and torch.equal(y[[0, 4]], clean[[0, 4]])
        got = hc.hc_layer_norm(x, quant=_dt("e4m3"), group=32)
        assert got["scale"][1:4].isnan().all() and not got["scale"][[0, 4]].isnan().any()


def test_in_place_given_outputs_and_no_rows():
    note("hc_layer_norm in place on the residual; T = 0")
    x, r = (torch.randn(9, 260, device="cuda").bfloat16() for _ in range(2))
    b = torch.randn(260, device="cuda")
    want = hc.hc_layer_norm(x, None, b, residual=r, quant=_dt("e4m3"), group=32)
    y, sc = torch.zeros(9, 260, dtype=_dt("e4m3"), device="cuda"), torch.zeros(9, 9, device="cuda")
    got = hc.hc_layer_norm(x, None, b, residual=r, s_out=r, quant=_dt("e4m3"), group=32, out=(y, sc))
    assert got["s"] is r and torch.equal(r, want["s"]) and torch.equal(y.view(torch.uint8), want["y"].view(torch.uint8))
    assert torch.equal(sc, want["scale"])
    e = torch.empty(0, 64, device="cuda")
    assert hc.hc_layer_norm(e, torch.ones(64, device="cuda"), residual=e)["s"].shape == (0, 64)
    dx, dw, db = hc.hc_layer_norm_backward(e, None, e)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_unaligned_arrays():
    note("hc_layer_norm on arrays one element off a 16-byte address")
    for dt in ("bf16", "f32"):
        big = torch.randn(2 * 520 + 9, device="cuda").to(_dt(dt))
        x = big[1:1 + 2 * 520].view(2, 520)
        assert x.data_ptr() % 16
        y = hc.hc_layer_norm(x)["y"]
        got = hc.hc_layer_norm_backward(x, None, y)
        want = hc.hc_layer_norm_backward(x.clone(), None, y)
        assert torch.equal(y, hc.hc_layer_norm(x.clone())["y"])
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_binding_refuses():
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: hc.hc_layer_norm(x.t()), lambda: hc.hc_layer_norm(x, w[:32]), lambda: hc.hc_layer_norm(x, w, w[:1]),
                lambda: hc.hc_layer_norm(x, w, w, residual=x[:2]), lambda: hc.hc_layer_norm(x, s_out=x),
                lambda: hc.hc_layer_norm(x, group=32), lambda: hc.hc_layer_norm(x, quant=_dt("i8"), group=48),
                lambda: hc.hc_layer_norm_backward(x, w, x[:2]), lambda: hc.hc_pre_layer_norm(x, w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: hc.hc_layer_norm(x.half()), lambda: hc.hc_layer_norm(x.cpu()), lambda: hc.hc_layer_norm(x, w.double()),
                lambda: hc.hc_layer_norm(x, w, w.bfloat16()), lambda: hc.hc_layer_norm(x, quant=torch.uint8),
                lambda: hc.hc_layer_norm_backward(x, w, x.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(hc.HCError):
        hc.hc_layer_norm(x, eps=-1.0)
