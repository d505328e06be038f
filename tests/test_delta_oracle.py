"""The gated delta rule's float64 form against closed forms and central differences, and the refusals of
its calls, found on the host before any device work (CPU)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import sublayer_ops as R


def _inputs(B=2, S=6, Hk=1, Hv=2, Dk=3, Dv=4, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.normal(size=(B, S, Hk, Dk)), rng.normal(size=(B, S, Hk, Dk)) / 2, rng.normal(size=(B, S, Hv, Dv)),
            -rng.uniform(0, 1, size=(B, S, Hv)), rng.uniform(0, 1, size=(B, S, Hv)), rng.normal(size=(B, Hv, Dk, Dv)))


def test_a_key_reads_back_what_it_wrote():
    """beta 1, no decay, unit keys: the state answers k_t with v_t, whatever it held before."""
    q, k, v, g, beta, M = _inputs()
    k = k / np.linalg.norm(k, axis=-1, keepdims=True)
    o, _ = R.gated_delta(k, k, v, 0 * g, np.ones_like(beta), M, scale=1.0)
    np.testing.assert_allclose(o, v, atol=1e-12)


def test_beta_zero_only_decays():
    q, k, v, g, beta, M = _inputs()
    _, last = R.gated_delta(q, k, v, g, 0 * beta, M)
    np.testing.assert_allclose(last, M * np.exp(g.sum(1))[:, :, None, None], atol=1e-14)


def test_orthogonal_keys_are_a_linear_attention():
    S = 4
    k = np.eye(S)[None, :, None]
    rng = np.random.default_rng(1)
    q, v = rng.normal(size=(1, S, 1, S)), rng.normal(size=(1, S, 1, 5))
    o, _ = R.gated_delta(q, k, v, np.zeros((1, S, 1)), np.ones((1, S, 1)), scale=1.0)
    want = np.tril(q[0, :, 0] @ k[0, :, 0].T) @ v[0, :, 0]
    np.testing.assert_allclose(o[0, :, 0], want, atol=1e-14)


def test_lengths_and_pieces():
    q, k, v, g, beta, M = _inputs()
    o, last = R.gated_delta(q, k, v, g, beta, M, lengths=[4, 0], o_init=np.full(v.shape, 7.0))
    a, m = R.gated_delta(q[:1, :2], k[:1, :2], v[:1, :2], g[:1, :2], beta[:1, :2], M[:1])
    b, m = R.gated_delta(q[:1, 2:4], k[:1, 2:4], v[:1, 2:4], g[:1, 2:4], beta[:1, 2:4], m)
    np.testing.assert_allclose(o[0, :4], np.concatenate([a, b], 1)[0], atol=1e-13)
    np.testing.assert_allclose(last[0], m[0], atol=1e-13)
    assert (o[0, 4:] == 7).all() and (o[1] == 7).all() and np.array_equal(last[1], M[1])


@pytest.mark.parametrize("lengths", [None, [6, 4]])
def test_backward_is_the_derivative(lengths):
    ins = _inputs(seed=2)
    rng = np.random.default_rng(3)
    do, dM = rng.normal(size=ins[2].shape), rng.normal(size=ins[5].shape)

    def loss(*x):
        o, M = R.gated_delta(*x, lengths=lengths)
        return (o * do).sum() + (M * dM).sum()

    q, k, v, g, beta, M = ins
    grads = R.gated_delta_backward(q, k, v, g, beta, do, M, dM, lengths)
    for i, (x, got) in enumerate(zip(ins, grads)):
        for at in [tuple(int(rng.integers(0, s)) for s in x.shape) for _ in range(12)]:
            p, m = [y.copy() for y in ins], [y.copy() for y in ins]
            p[i][at] += 1e-6
            m[i][at] -= 1e-6
            np.testing.assert_allclose(got[at], (loss(*p) - loss(*m)) / 2e-6, rtol=1e-5, atol=1e-7)


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


def test_forward_refusals(L):
    ws = L.hc_gated_delta_workspace_bytes
    for bad in ((-1, 8, 1, 1, 8, 8, 1), (1, -1, 1, 1, 8, 8, 1), (1, 8, 0, 0, 8, 8, 1), (1, 8, 2, 3, 8, 8, 1),
                (1, 8, 2, 0, 8, 8, 1), (1, 8, 1, 1, 0, 8, 1), (1, 8, 1, 1, 257, 8, 1), (1, 8, 1, 1, 8, 257, 1),
                (1, 8, 1, 1, 8, 0, 1), (1, 8, 1, 1, 8, 8, 2), (1 << 20, 1, 1, 1, 8, 8, 1), (1, 1 << 30, 1, 1, 8, 8, 1),
                (1, 1, 1, 1 << 20, 8, 8, 1), (1 << 40, 1, 1, 1 << 40, 8, 8, 1), (1, 1 << 62, 1, 1, 8, 8, 1)):
        assert ws(*bad) == -1, bad
    assert ws(0, 300, 1, 1, 8, 8, 1) == 0 and ws(4, 1, 1, 1, 8, 8, 1) == 0
    need = ws(2, 300, 1, 2, 32, 32, 1)
    assert need > 0

    def fwd(q=at(0), k=at(1), v=at(2), dt=1, B=2, S=300, Hk=1, Hv=2, Dk=32, Dv=32, g=at(3), be=at(4), s0=at(5),
            ln=at(6), o=at(7), s1=at(8), w=at(9), wb=need):
        return L.hc_gated_delta(q, k, v, dt, B, S, Hk, Hv, Dk, Dv, g, be, 1.0, s0, ln, o, s1, w, wb, None)

    assert fwd(dt=2) == -3 and fwd(B=-1) == -2 and fwd(S=-1) == -2 and fwd(Hv=3, Hk=2) == -2 and fwd(Dk=257) == -2
    for name in ("q", "k", "v", "g", "be", "o"):
        assert fwd(**{name: None}) == -1, name
    for name in ("q", "o", "be", "s0", "ln", "s1"):
        assert fwd(**{name: ctypes.c_void_p(FAKE + 1)}) == -4, name
    assert fwd(w=None) == -8 and fwd(wb=need - 1) == -8 and fwd(w=ctypes.c_void_p(at(9).value + 16)) == -8
    for x in (0, 1, 2, 3, 4, 5, 6):
        assert fwd(o=at(x)) == -5, x
        assert fwd(w=at(x)) == -5, x
        if x != 5:
            assert fwd(s1=at(x)) == -5, x
    assert fwd(s1=at(7)) == -5 and fwd(s1=ctypes.c_void_p(at(5).value + 4)) == -5
    assert fwd(B=0, q=None, k=None, v=None, g=None, be=None, o=None, w=None, wb=0) == 0
    assert fwd(S=0, q=None, k=None, v=None, g=None, be=None, o=None, s1=None, w=None, wb=0) == 0


def test_backward_refusals(L):
    ws = L.hc_gated_delta_backward_workspace_bytes
    assert ws(1, 8, 2, 3, 8, 8, 1) == -1 and ws(1, 8, 1, 1, 257, 8, 1) == -1 and ws(1, 8, 1, 1, 8, 8, 7) == -1
    assert ws(0, 8, 1, 1, 8, 8, 1) == 0 and ws(1, 0, 1, 1, 8, 8, 1) == 0
    need = ws(2, 30, 1, 2, 32, 32, 1)
    assert need > 0

    def bwd(q=at(0), k=at(1), v=at(2), d=at(3), dt=1, B=2, S=30, Hk=1, Hv=2, Dk=32, Dv=32, g=at(4), be=at(5), s0=at(6),
            s1=at(7), ln=at(8), dq=at(9), dk=at(10), dv=at(11), dg=at(12), db=at(13), d0=at(14), w=at(20), wb=need):
        return L.hc_gated_delta_backward(q, k, v, d, dt, B, S, Hk, Hv, Dk, Dv, g, be, 1.0, s0, s1, ln, dq, dk, dv, dg,
                                         db, d0, w, wb, None)

    assert bwd(dt=3) == -3 and bwd(Hv=3, Hk=2) == -2 and bwd(S=-1) == -2
    for name in ("q", "k", "v", "d", "g", "be", "dq", "dk", "dv", "dg", "db"):
        assert bwd(**{name: None}) == -1, name
    for name in ("k", "d", "s1", "dg", "d0"):
        assert bwd(**{name: ctypes.c_void_p(FAKE + 1)}) == -4, name
    assert bwd(w=None) == -8 and bwd(wb=need - 1) == -8
    for x in range(9):
        for name in ("dq", "dk", "dv", "dg", "db", "d0", "w"):
            assert bwd(**{name: at(x)}) == -5, (name, x)
    assert bwd(dk=at(9)) == -5 and bwd(d0=at(12)) == -5 and bwd(w=at(11)) == -5
    assert bwd(B=0, q=None, k=None, v=None, d=None, g=None, be=None, dq=None, dk=None, dv=None, dg=None, db=None, w=None,
               wb=0) == 0
