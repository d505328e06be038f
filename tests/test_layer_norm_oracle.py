"""The layer norm's float64 form against closed forms and central differences, and the refusals of its
calls, found on the host before any device work (CPU)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import sublayer_ops as R


def test_closed_form_and_equal_values():
    v = np.array([[1.0, 3.0, 1.0, 3.0], [5.0, 5.0, 5.0, 5.0]])
    y = R.layer_norm(v, [1, 1, 2, 2], [0, 1, 0, 1], 0.0)
    np.testing.assert_allclose(y, [[-1, 2, -2, 3], [0, 1, 0, 1]], atol=1e-15)


def test_does_not_see_a_shift():
    v = np.random.default_rng(0).normal(size=(3, 50))
    np.testing.assert_allclose(R.layer_norm(v + 1000, None, None, 1e-5), R.layer_norm(v, None, None, 1e-5), atol=1e-11)


def test_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    v, w, b, dy, ds = (rng.normal(size=s) for s in ((3, 7), 7, 7, (3, 7), (3, 7)))
    dx, dw, db = R.layer_norm_backward(v, w, 0.1, dy, ds)

    def diff(f, x):
        out = np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            p, q = x.copy(), x.copy()
            p[i] += 1e-6
            q[i] -= 1e-6
            out[i] = (f(p) - f(q)) / 2e-6
        return out

    np.testing.assert_allclose(dx, diff(lambda x: (R.layer_norm(x, w, b, 0.1) * dy).sum() + (x * ds).sum(), v),
                               rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, diff(lambda x: (R.layer_norm(v, x, b, 0.1) * dy).sum(), w), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(db, diff(lambda x: (R.layer_norm(v, w, x, 0.1) * dy).sum(), b), rtol=1e-6, atol=1e-8)


FAKE = 0x10000


def at(i):
    """The i-th of a row of made-up addresses 1 MiB apart (never dereferenced)."""
    return ctypes.c_void_p(0x10000000 + (i << 20))


@pytest.fixture(scope="module")
def L():
    import stream_residual_mixing_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.fail("libhc.so is not built (run __graft_entry__.build())")
    return m.lib()


def test_refusals(L):
    def norm(x=at(0), dt=1, T=8, C=64, res=at(1), w=at(2), b=at(3), eps=1e-6, s=at(4), ydt=1, group=0, y=at(5),
             sc=None):
        return L.hc_layer_norm(x, dt, T, C, res, w, b, eps, s, ydt, group, y, sc, None)

    assert norm(dt=7) == -3 and norm(ydt=0) == -3 and norm(ydt=5) == -3
    assert norm(T=-1) == -2 and norm(C=0) == -2 and norm(C=16385) == -2
    assert norm(eps=-1.0) == -2 and norm(eps=float("nan")) == -2 and norm(eps=float("inf")) == -2
    assert norm(group=32) == -2 and norm(ydt=2, group=16, sc=at(6)) == -2
    assert norm(x=None) == -1 and norm(y=None) == -1 and norm(res=None) == -1 and norm(ydt=2) == -1
    assert norm(x=ctypes.c_void_p(FAKE + 1)) == -4 and norm(b=ctypes.c_void_p(FAKE + 2)) == -4
    assert norm(y=at(0)) == -5 and norm(y=at(1)) == -5 and norm(y=at(3)) == -5 and norm(s=at(0)) == -5
    assert norm(y=at(4)) == -5 and norm(s=at(3)) == -5 and norm(s=ctypes.c_void_p(at(1).value + 2)) == -5
    assert norm(T=0, x=None, y=None, res=None, s=None) == 0

    def pre(n=4, h=at(1), F=at(2), y=at(3), X=at(0), b=at(4)):
        return L.hc_pre_layer_norm(X, 1, 8, n, 64, h, None, b, 1e-6, F, 1, 0, y, None, None)

    assert pre(n=0) == -2 and pre(n=65) == -2 and pre(h=None) == -1 and pre(X=None) == -1
    assert pre(F=at(3)) == -5 and pre(y=at(0)) == -5 and pre(F=at(1)) == -5 and pre(b=at(3)) == -5

    assert L.hc_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert L.hc_layer_norm_backward_workspace_bytes(8, 0) == -1 and L.hc_layer_norm_backward_workspace_bytes(-1, 8) == -1
    need = L.hc_layer_norm_backward_workspace_bytes(8, 64)
    assert need > 0

    def bwd(s=at(0), dt=1, T=8, C=64, w=at(1), eps=1e-6, dy=at(2), ds=at(3), dx=at(4), dw=at(5), db=at(6), ws=at(7),
            wsb=need):
        return L.hc_layer_norm_backward(s, dt, T, C, w, eps, dy, ds, dx, dw, db, ws, wsb, None)

    assert bwd(dt=2) == -3 and bwd(C=20000) == -2 and bwd(eps=-1.0) == -2
    assert bwd(s=None) == -1 and bwd(dy=None) == -1 and bwd(dx=None) == -1
    assert bwd(db=ctypes.c_void_p(FAKE + 2)) == -4
    assert bwd(ws=None) == -8 and bwd(wsb=need - 1) == -8 and bwd(ws=ctypes.c_void_p(at(7).value + 16)) == -8
    assert bwd(dw=None, wsb=need - 1) == -8  # one of the two sums alone needs it as well
    assert bwd(dx=at(0)) == -5 and bwd(dx=at(2)) == -5 and bwd(dw=at(3)) == -5 and bwd(db=at(4)) == -5
    assert bwd(db=at(5)) == -5 and bwd(dx=ctypes.c_void_p(at(3).value + 2)) == -5 and bwd(ws=at(6)) == -5
    assert bwd(T=0, s=None, dy=None, dx=None, dw=None, db=None, ws=None, wsb=0) == 0
