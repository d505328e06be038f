"""The float64 forms of oracle/sublayer_ops.py against closed forms and central differences (CPU)."""
import numpy as np
import pytest

from oracle import sublayer_ops as R


def _diff(f, x, seed=0, n=6):
    """Central differences of the scalar f at n entries of x: (indices, values)."""
    rng = np.random.default_rng(seed)
    flat = [tuple(int(rng.integers(0, s)) for s in x.shape) for _ in range(n)]
    out = []
    for i in flat:
        h = 1e-6
        p, q = x.copy(), x.copy()
        p[i] += h
        q[i] -= h
        out.append((f(p) - f(q)) / (2 * h))
    return flat, np.array(out)


def test_norm_closed_form_and_zero_row():
    v = np.array([[3.0, -3.0, 3.0, -3.0], [0.0, 0.0, 0.0, 0.0]])
    y = R.rms_norm(v, None, 0.0)
    np.testing.assert_allclose(y[0], np.sign(v[0]), atol=1e-15)
    assert not y[1].any()


def test_norm_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    v, w, dy, ds = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dx, dw = R.rms_norm_backward(v, w, 0.1, dy, ds)
    at, d = _diff(lambda p: (R.rms_norm(p, w, 0.1) * dy).sum() + (p * ds).sum(), v)
    np.testing.assert_allclose([dx[i] for i in at], d, rtol=1e-6, atol=1e-8)
    at, d = _diff(lambda p: (R.rms_norm(v, p, 0.1) * dy).sum(), w)
    np.testing.assert_allclose([dw[i] for i in at], d, rtol=1e-6, atol=1e-8)


def test_scales_of_groups_with_a_short_last_one():
    y = np.array([[1.0, -4.48, 2.0, 0.0, 0.0]])
    np.testing.assert_allclose(R.quant_scales(y, "e4m3", 2), [[0.01, 2 / 448, 1.0]])
    assert R.per_channel(np.array([[1.0, 2.0, 3.0]]), 5, 2).tolist() == [[1, 1, 2, 2, 3]]


def test_scan_with_constant_gate_is_a_geometric_mean():
    g = np.full((1, 50, 1), np.log(3.0))  # a = 3/4
    y, h = R.gated_scan(np.ones((1, 50, 1)), g, tied=True)
    np.testing.assert_allclose(y[0, :, 0], 1 - 0.75 ** np.arange(1, 51), rtol=1e-14)
    y, h = R.gated_scan(np.ones((1, 50, 1)), g, np.full((1, 1), 4.0), tied=False)
    np.testing.assert_allclose(h, 4.0, rtol=1e-14)


@pytest.mark.parametrize("tied", [True, False])
def test_scan_backward_is_the_derivative(tied):
    rng = np.random.default_rng(2)
    B, S, C, L = 2, 6, 3, [6, 4]
    x, g, h0 = rng.normal(size=(B, S, C)), rng.normal(size=(B, S, C)), rng.normal(size=(B, C))
    dy, dl = rng.normal(size=(B, S, C)), rng.normal(size=(B, C))
    live = np.arange(S)[None, :, None] < np.array(L)[:, None, None]

    def f(x, g, h0):
        y, h = R.gated_scan(x, g, h0, L, tied)
        return (y * dy * live).sum() + (h * dl).sum()

    y, _ = R.gated_scan(x, g, h0, L, tied)
    dx, dg, dh0 = R.gated_scan_backward(x, g, y, dy, h0, dl, L, tied)
    for got, arr, fn in ((dx, x, lambda p: f(p, g, h0)), (dg, g, lambda p: f(x, p, h0)),
                         (dh0, h0, lambda p: f(x, g, p))):
        at, d = _diff(fn, arr, n=10)
        np.testing.assert_allclose([got[i] for i in at], d, rtol=1e-5, atol=1e-8)


def test_balance_loss_of_an_even_choice_is_coef():
    N, m, k, S = 6, 2, 3, 8
    idx = np.array([[0, 1, 2 + t % 4] for t in range(S)])
    r = R.balance_loss(np.full((S, 4), 0.3), idx, 1, S, N, m, coef=0.7)
    assert abs(r["loss"] - 0.7) < 1e-15 and r["count"].tolist() == [[8, 8, 2, 2, 2, 2]]
    assert R.balance_loss(np.full((S, 4), 0.3), idx, 1, S, N, m, mask=np.zeros(S))["loss"] == 0.0


def test_balance_backward_is_the_derivative_with_counts_held():
    rng = np.random.default_rng(3)
    B, S, N, m, k = 2, 5, 7, 2, 4
    score = rng.uniform(0.05, 0.95, size=(B * S, N - m))
    idx = np.sort(np.concatenate([np.tile([0, 1], (B * S, 1)), 2 + np.argsort(rng.random((B * S, 5)))[:, :2]], 1), 1)
    mask = rng.random(B * S) < 0.7
    r = R.balance_loss(score, idx, B, S, N, m, 0.3, mask)
    d = R.balance_loss_backward(score, r["count"], r["tokens"], k, B, S, N, m, 0.3, 2.0, mask)
    at, num = _diff(lambda p: 2.0 * R.balance_loss(p, idx, B, S, N, m, 0.3, mask)["loss"], score, n=12)
    np.testing.assert_allclose([d[i] for i in at], num, rtol=1e-5, atol=1e-9)


def test_router_backward_is_the_derivative():
    rng = np.random.default_rng(4)
    T, N, C, E = 3, 4, 5, 2
    X, w, ds = rng.normal(size=(T, N, C)), 0.3 * rng.normal(size=(N * C, E)), rng.normal(size=(T, E))

    def scores(X, w):
        x = X.reshape(T, -1)
        return R.sigmoid((x @ w) / np.sqrt((x * x).mean(1, keepdims=True)))

    out, dw = R.router_backward(X, w, scores(X, w), ds, np.zeros_like(X))
    at, d = _diff(lambda p: (scores(p, w) * ds).sum(), X, n=10)
    np.testing.assert_allclose([out[i] for i in at], d, rtol=1e-5, atol=1e-9)
    at, d = _diff(lambda p: (scores(X, p) * ds).sum(), w, n=10)
    np.testing.assert_allclose([dw[i] for i in at], d, rtol=1e-5, atol=1e-9)


def test_router_backward_skips_a_token_without_gradient():
    X = np.full((1, 2, 3), np.nan)
    out, dw = R.router_backward(X, np.ones((6, 1)), np.array([[np.nan]]), np.zeros((1, 1)), np.ones((1, 2, 3)))
    assert (out == 1).all() and not dw.any()
