"""CPU tests of the refusals of the norm, scan, balance-loss and router-backward calls:
each is found on the host, before any device work (no compute call is made here)."""
import ctypes
import os

import pytest

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


def test_norm_refusals(L):
    def norm(x=at(0), dt=1, T=8, C=64, res=at(1), w=at(2), eps=1e-6, s=at(3), ydt=1, group=0, y=at(4), sc=None):
        return L.hc_rms_norm(x, dt, T, C, res, w, eps, s, ydt, group, y, sc, None)

    assert norm(dt=7) == -3 and norm(ydt=0) == -3 and norm(ydt=5) == -3
    assert norm(T=-1) == -2 and norm(C=0) == -2 and norm(C=16385) == -2
    assert norm(eps=-1.0) == -2 and norm(eps=float("nan")) == -2 and norm(eps=float("inf")) == -2
    assert norm(group=32) == -2 and norm(ydt=2, group=16, sc=at(5)) == -2
    assert norm(x=None) == -1 and norm(y=None) == -1 and norm(res=None) == -1 and norm(ydt=2) == -1
    assert norm(x=ctypes.c_void_p(FAKE + 1)) == -4 and norm(ydt=3, sc=ctypes.c_void_p(FAKE + 2)) == -4
    assert norm(y=at(0)) == -5 and norm(y=at(1)) == -5 and norm(s=at(0)) == -5 and norm(y=at(3)) == -5
    assert norm(s=ctypes.c_void_p(at(1).value + 2)) == -5 and norm(ydt=2, sc=at(4)) == -5
    assert norm(T=0, x=None, y=None, res=None, s=None) == 0

    def pre(n=4, h=at(1), F=at(2), y=at(3), X=at(0)):
        return L.hc_pre_norm(X, 1, 8, n, 64, h, None, 1e-6, F, 1, 0, y, None, None)

    assert pre(n=0) == -2 and pre(n=65) == -2 and pre(h=None) == -1 and pre(X=None) == -1
    assert pre(F=at(3)) == -5 and pre(y=at(0)) == -5 and pre(F=at(1)) == -5

    assert L.hc_rms_norm_backward_workspace_bytes(0, 64) == 0
    assert L.hc_rms_norm_backward_workspace_bytes(8, 0) == -1
    need = L.hc_rms_norm_backward_workspace_bytes(8, 64)
    assert need > 0

    def bwd(s=at(0), dt=1, T=8, C=64, w=at(1), eps=1e-6, dy=at(2), ds=at(3), dx=at(4), dw=at(5), ws=at(6), wsb=need):
        return L.hc_rms_norm_backward(s, dt, T, C, w, eps, dy, ds, dx, dw, ws, wsb, None)

    assert bwd(dt=2) == -3 and bwd(C=20000) == -2 and bwd(eps=-1.0) == -2
    assert bwd(s=None) == -1 and bwd(dy=None) == -1 and bwd(dx=None) == -1
    assert bwd(dw=ctypes.c_void_p(FAKE + 2)) == -4
    assert bwd(ws=None) == -8 and bwd(wsb=need - 1) == -8 and bwd(ws=ctypes.c_void_p(at(6).value + 16)) == -8
    assert bwd(dx=at(0)) == -5 and bwd(dx=at(2)) == -5 and bwd(dw=at(3)) == -5 and bwd(dw=at(4)) == -5
    assert bwd(dx=ctypes.c_void_p(at(3).value + 2)) == -5 and bwd(ws=at(4)) == -5
    assert bwd(T=0, s=None, dy=None, dx=None, dw=None, ws=None, wsb=0) == 0


def test_scan_refusals(L):
    assert L.hc_gated_scan_workspace_bytes(-1, 8, 64) == -1 and L.hc_gated_scan_workspace_bytes(1, 8, 0) == -1
    assert L.hc_gated_scan_workspace_bytes(1 << 20, 1 << 20, 64) == -1
    assert L.hc_gated_scan_workspace_bytes(0, 8, 64) == 0
    need = L.hc_gated_scan_workspace_bytes(2, 300, 64)

    def fwd(x=at(0), g=at(1), dt=1, B=2, S=300, C=64, h0=at(2), ln=at(3), y=at(4), h=at(5), ws=at(6), wsb=need):
        return L.hc_gated_scan(x, g, dt, B, S, C, h0, ln, 1, y, h, ws, wsb, None)

    assert fwd(dt=2) == -3 and fwd(B=-1) == -2 and fwd(S=-1) == -2 and fwd(C=0) == -2
    assert fwd(x=None) == -1 and fwd(g=None) == -1 and fwd(y=None) == -1
    assert fwd(x=ctypes.c_void_p(FAKE + 1)) == -4 and fwd(ln=ctypes.c_void_p(FAKE + 2)) == -4
    if need:
        assert fwd(ws=None) == -8 and fwd(wsb=need - 1) == -8 and fwd(ws=at(4)) == -5
    assert fwd(y=at(0)) == -5 and fwd(y=at(1)) == -5 and fwd(y=at(2)) == -5 and fwd(h=at(3)) == -5
    assert fwd(h=at(4)) == -5 and fwd(h=ctypes.c_void_p(at(2).value + 4)) == -5
    assert fwd(B=0, x=None, g=None, y=None, ws=None, wsb=0) == 0
    assert fwd(S=0, x=None, g=None, y=None, h=None, ws=None, wsb=0) == 0

    def bwd(x=at(0), g=at(1), y=at(2), dy=at(3), dt=1, h0=at(4), dl=at(5), dx=at(6), dg=at(7), d0=at(8), ws=at(9),
            wsb=need):
        return L.hc_gated_scan_backward(x, g, y, dy, dt, 2, 300, 64, h0, dl, None, 1, dx, dg, d0, ws, wsb, None)

    assert bwd(dt=3) == -3 and bwd(y=None) == -1 and bwd(dy=None) == -1 and bwd(dx=None) == -1 and bwd(dg=None) == -1
    if need:
        assert bwd(wsb=0) == -8
    assert bwd(dx=at(3)) == -5 and bwd(dg=at(2)) == -5 and bwd(dx=at(7)) == -5 and bwd(d0=at(5)) == -5
    assert bwd(d0=at(4)) == -5


def test_router_refusals(L):
    need = L.xhc_balance_loss_workspace_bytes(2, 9000, 16, 2)
    assert need > 0 and L.xhc_balance_loss_workspace_bytes(1, 509, 8, 1) == 0  # one workgroup takes those alone
    assert L.xhc_balance_loss_workspace_bytes(2, 300, 65, 2) == -1
    assert L.xhc_balance_loss_workspace_bytes(1 << 20, 1 << 20, 16, 2) == -1

    def loss(s=at(0), i=at(1), mk=at(2), B=2, S=9000, N=16, k=4, m=2, lo=at(3), c=at(4), t=at(5), p=at(6), ws=at(7),
             wsb=need):
        return L.xhc_balance_loss(s, i, mk, B, S, N, k, m, 0.01, lo, c, t, p, ws, wsb, None)

    assert loss(m=0) == -2 and loss(k=2) == -2 and loss(N=3) == -2 and loss(N=65) == -2 and loss(k=17, N=32) == -2
    assert loss(B=-1) == -2 and loss(S=1 << 26) == -2
    assert loss(s=None) == -1 and loss(i=None) == -1 and loss(lo=None) == -1 and loss(p=None) == -1
    assert loss(s=ctypes.c_void_p(FAKE + 1)) == -4
    assert loss(ws=None) == -8 and loss(wsb=need - 1) == -8
    assert loss(lo=at(0)) == -5 and loss(c=at(5)) == -5 and loss(p=at(2)) == -5 and loss(ws=at(1)) == -5

    def bwd(s=at(0), c=at(1), t=at(2), mk=None, dl=at(3), d=at(4), k=4, m=2):
        return L.xhc_balance_loss_backward(s, c, t, mk, 2, 300, 16, k, m, 0.01, dl, d, None)

    assert bwd(k=2) == -2 and bwd(c=None) == -1 and bwd(t=None) == -1 and bwd(d=None) == -1
    assert bwd(d=at(0)) == -5 and bwd(d=at(3)) == -5

    need = L.xhc_router_backward_workspace_bytes(8, 16, 64, 2, 1)
    assert need > 0 and L.xhc_router_backward_workspace_bytes(0, 16, 64, 2, 1) == 0
    for bad in ((8, 17, 64, 2, 1), (8, 16, 60, 2, 1), (8, 2, 64, 2, 1), (8, 16, 64, 0, 1), (1 << 24, 16, 64, 2, 1),
                (8, 16, 64, 2, 0)):
        assert L.xhc_router_backward_workspace_bytes(*bad) == -1

    def rt(X=at(0), dt=1, T=8, N=16, C=64, m=2, w=at(1), s=at(2), d=at(3), dX=at(4), o=at(5), dw=at(6), ws=at(7),
           wsb=need):
        return L.xhc_router_backward(X, dt, T, N, C, m, w, s, d, dX, o, dw, ws, wsb, None)

    assert rt(dt=0) == -3 and rt(N=17) == -2 and rt(C=48) == -2 and rt(m=16) == -2 and rt(T=-1) == -2
    assert rt(X=None) == -1 and rt(dX=None) == -1 and rt(o=None) == -1 and rt(dw=None) == -1 and rt(s=None) == -1
    assert rt(X=ctypes.c_void_p(FAKE + 8)) == -4 and rt(w=ctypes.c_void_p(FAKE + 2)) == -4
    assert rt(ws=None) == -8 and rt(wsb=need - 1) == -8
    assert rt(o=at(0)) == -5 and rt(dw=at(4)) == -5 and rt(dw=at(1)) == -5
    assert rt(o=ctypes.c_void_p(at(4).value + 16)) == -5 and rt(ws=at(5)) == -5


def test_sizes_whose_grids_no_launch_takes(L):
    """A launch has fewer than 2^32 threads along x: calls that would need more are refused."""
    ws = L.xhc_router_backward_workspace_bytes
    assert ws((1 << 24) - 32, 2, 32, 1, 1) > 0
    for T in ((1 << 24) - 31, (1 << 24) - 1):  # whole groups of 32 tokens, 256 threads each token: 2^32
        assert ws(T, 2, 32, 1, 1) == -1
    ws = L.xhc_balance_loss_workspace_bytes
    assert ws(1, (1 << 26) - 4, 32, 2) > 0 and ws((1 << 24) - 1, 1, 16, 2) > 0
    assert ws(1, (1 << 26) - 3, 32, 2) == -1  # 64 threads a token, workgroups of 256
    assert ws(1 << 24, 1, 16, 2) == -1 and ws(1 << 25, 0, 16, 2) == -1  # a workgroup a sequence

    def bwd(B, S):
        return L.xhc_balance_loss_backward(None, None, None, None, B, S, 32, 4, 2, 0.01, None, None, None)

    assert bwd(1, (1 << 26) - 3) == -2 and bwd(1 << 24, 1) == -2 and bwd(1, (1 << 26) - 4) == -1
