"""The gated delta rule's backward on the GPU against its float64 form (oracle/sublayer_ops.py).

Bounds are on norms for each head, as in test_gpu_delta.py: _bounds() follows the chunks' products
forward and back, each off by c = 2^-15 of its terms' magnitudes and passing on its operands'
errors times the other operand's norm. The maps of a state over whole chunks have no norm above 1
(unit keys, 0 <= beta <= 1). The running sum that makes dg of a chunk's 64 terms has a norm of
at most 64. A bfloat16 output rounds by 2^-8 of each element; where value heads share a key head its
bound is the sum of theirs.
"""
import numpy as np
import pytest

from hc_testutil import have_gpu, note
from oracle import sublayer_ops as R
from test_gpu_delta import C15, P, _norm, _two, down, inputs, up

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate0")


def _bounds(q, k, v, g, beta, do, M, N, scale, n):
    """Bounds on the norms of the errors of one head's six gradients, n tokens."""
    ab, keep, em = np.abs, [], 0.0
    for t in range(0, n, 64):
        at = slice(t, min(n, t + 64))
        Q, K, V, G, b, d = q[at], k[at], v[at], np.cumsum(g[at]), beta[at][:, None], scale * do[at]
        one = np.eye(len(G))
        D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
        kk, Pm = np.tril(D * (K @ K.T), -1), D * (Q @ K.T)
        A = kk * b.T
        T = np.linalg.inv(one + A)
        aT = ab(T) @ (one + ab(A)) @ ab(T) + ab(T)  # |T| with the error of its own making
        ahead, end = np.exp(G)[:, None], np.exp(G[-1] - G)[:, None]
        r = V - ahead * (K @ M)
        z = T @ r
        ez = _two(T) * (C15 * _norm(ab(V) + ahead * (ab(K) @ ab(M))) + _norm(K) * em) + C15 * _norm(aT @ ab(r))
        keep.append((Q, K, b, d, D, kk, Pm, T, aT, ahead, end, M, em, z, ez))
        x = b * z
        em = em + _two(K * end) * (b.max() * ez) + C15 * _norm(ab(M) + ab(K * end).T @ ab(x))
        M = np.exp(G[-1]) * M + (K * end).T @ x
    out, en = np.zeros(6), 0.0
    for Q, K, b, d, D, kk, Pm, T, aT, ahead, end, M, em, z, ez in reversed(keep):
        x, ex = b * z, b.max() * ez
        aP = ab(Pm) + D * (ab(Q) @ ab(K).T)
        dx = Pm.T @ d + end * (K @ N)
        edx = _two(K * end) * en + C15 * _norm(aP.T @ ab(d) + end * (ab(K) @ ab(N)))
        w = T.T @ (b * dx)
        ew = _two(T) * edx + C15 * _norm(aT.T @ ab(b * dx))
        B, Am = np.tril(d @ x.T) * D, np.tril(w @ x.T, -1) * D
        eB = _two(d) * ex + C15 * _norm(np.tril(ab(d) @ ab(x).T) * D)
        eA = _two(w) * ex + _two(x) * ew + C15 * _norm(np.tril(ab(w) @ ab(x).T) * D)
        eq = _two(d) * em + _two(K) * eB + C15 * _norm(ahead * (ab(d) @ ab(M).T) + ab(B) @ ab(K))
        eread = _two(w) * em + _norm(M) * ew + _two(K) * eA + C15 * _norm(ahead * (ab(w) @ ab(M).T) + ab(Am) @ ab(K))
        eearly = _two(x) * en + _norm(N) * ex + C15 * _norm(end * (ab(x) @ ab(N).T))
        ewrite = eearly + _two(Q) * eB + _two(K) * eA + C15 * _norm(ab(B).T @ ab(Q) + ab(Am).T @ ab(K))
        eb = _norm(dx) * ez + _norm(z) * edx + _two(w) * ez + _two(z) * ew + \
            C15 * _norm((ab(z) * ab(dx)).sum(1) + (np.tril(D, -1) * (ab(K) @ ab(K).T) * (ab(w) @ ab(z).T)).sum(0)) + \
            C15 * _norm((D * (ab(Q) @ ab(K).T) * (ab(d) @ ab(z).T)).sum(0) + end[:, 0] * (ab(K) * (ab(z) @ ab(N).T)).sum(1))
        eG = eq + eread + ewrite
        eend = np.sqrt(len(K)) * eearly + em * _norm(N) + en * _norm(M) + C15 * _norm(M) * _norm(N)
        eg = 64 * eG + 8 * eend
        for i, e in enumerate((eq, eread + ewrite, ew, eg, eb)):
            out[i] += e * e
        en = en + _two(K * ahead) * ew + C15 * _norm(ab(N) + ab(Q * ahead).T @ ab(d) + ab(K * ahead).T @ ab(w))
        N = ahead[-1, 0] * N + (Q * ahead).T @ d - (K * ahead).T @ w
    return np.append(np.sqrt(out[:5]), en)


def check_backward(got, ins, do, dstate, lengths, dt, scale=None, slack=1):
    q, k, v, g, beta, M, do, dM = (down(x) for x in (*ins, do, dstate))
    B, S, Hk, Dk = q.shape
    Hv = v.shape[2]
    scale = Dk ** -0.5 if scale is None else scale
    ref = R.gated_delta_backward(q, k, v, g, beta, do, M, dM, lengths, scale)
    for b in range(B):
        n = S if lengths is None else int(np.clip(lengths[b], 0, S))
        shared = np.zeros((Hk, 2))
        for h in range(Hv):
            kh = h // (Hv // Hk)
            e = _bounds(q[b, :, kh], k[b, :, kh], v[b, :, h], g[b, :, h], beta[b, :, h], do[b, :, h], M[b, h], dM[b, h],
                        scale, n) * slack
            shared[kh] += e[:2]
            for i, rnd in ((2, P[dt]), (3, 2.0 ** -22), (4, 2.0 ** -22), (5, 2.0 ** -22)):
                x, y = (down(got[i])[b, h], ref[i][b, h]) if i == 5 else (down(got[i])[b, :, h], ref[i][b, :, h])
                _close(NAMES[i], (b, h), x, y, rnd, e[i])
        for kh in range(Hk):
            for i in (0, 1):
                _close(NAMES[i], (b, kh), down(got[i])[b, :, kh], ref[i][b, :, kh], P[dt] + 2.0 ** -22, shared[kh, i])
        for t in got[:5]:
            assert not t[b, n:].any(), "a token behind the length has a gradient"


def _close(name, where, x, y, rnd, bound):
    assert np.isfinite(x).all(), (name, where)
    err = np.abs(x - y)
    more = _norm(np.maximum(err - rnd * (np.abs(y) + err), 0))
    assert more <= bound, (name, where, more, bound)


SIZES = [(1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 128, 128), (2, 5, 1, 3, 100, 36), (1, 9, 1, 1, 64, 64), (1, 63, 1, 2, 24, 40),
         (2, 64, 2, 2, 128, 64), (1, 65, 1, 1, 128, 128), (2, 150, 1, 3, 72, 100), (1, 129, 1, 1, 200, 30),
         (1, 130, 1, 2, 256, 256), (1, 70, 2, 2, 33, 17), (1, 130, 1, 1, 7, 130), (1, 100, 1, 2, 129, 64),
         (1, 400, 1, 1, 64, 128)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward(size, dt):
    B, S, Hk, Hv, Dk, Dv = size
    rng = np.random.default_rng(S)
    ins = inputs(*size, dt, seed=S + Dk)
    do, dM = up(rng.normal(size=(B, S, Hv, Dv)), dt), up(rng.normal(size=(B, Hv, Dk, Dv)))
    for L in (None, rng.integers(0, S + 1, size=B)):
        note(f"hc_gated_delta_backward {size} {dt} lengths={L}")
        lengths = None if L is None else torch.from_numpy(L.astype(np.int32)).cuda()
        got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM, lengths=lengths)
        torch.cuda.synchronize()
        check_backward(got, ins, do, dM, L, dt)


@pytest.mark.parametrize("size", [(3, 1100, 1, 1, 64, 24), (2, 1024, 1, 2, 40, 80), (1, 1030, 1, 1, 130, 66)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_segments(size, dt):
    """Few heads and long sequences are walked in segments: as in the forward's test, with twice the bounds."""
    B, S, Hk, Hv, Dk, Dv = size
    ins = inputs(*size, dt, seed=S)
    rng = np.random.default_rng(S)
    do, dM = up(rng.normal(size=(B, S, Hv, Dv)), dt), up(rng.normal(size=(B, Hv, Dk, Dv)))
    ends = [S, 256, 0, 257, 700, 1]
    for turn in range(0, len(ends), B):
        L = np.array((ends[turn:] + ends)[:B])
        note(f"hc_gated_delta_backward {size} {dt} lengths={L}")
        got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM, lengths=torch.from_numpy(L.astype(np.int32)).cuda())
        torch.cuda.synchronize()
        check_backward(got, ins, do, dM, L, dt, slack=2)


def test_against_differences_of_the_forward():
    """A step along a random direction of every input, in float32: the forward's loss differences against
    the gradients. With steps of 2^-6 the difference's own error is the third derivative's 2^-12 of
    the values and the loss's 2^-15 over the step: 2^-8 of the norms' product is above both."""
    note("hc_gated_delta_backward against differences")
    ins = inputs(2, 100, 1, 2, 32, 24, "f32", seed=11)
    rng = np.random.default_rng(12)
    do, dM = up(rng.normal(size=(2, 100, 2, 24))), up(rng.normal(size=(2, 2, 32, 24)))
    got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM)

    def loss(x):
        o, M = hc.hc_gated_delta(*x)
        return float((o.double() * do.double()).sum() + (M.double() * dM.double()).sum())

    for i in range(6):
        way = torch.from_numpy(rng.normal(size=tuple(ins[i].shape)).astype(np.float32)).cuda()
        if i == 3:
            way = -way.abs() * 0.1
        way = way / way.norm()
        p, m = list(ins), list(ins)
        p[i], m[i] = ins[i] + way / 64, ins[i] - way / 64
        slope = (loss(p) - loss(m)) * 32
        want = float((got[i].double() * way.double()).sum())
        assert abs(slope - want) <= 2.0 ** -8 * float(got[i].double().norm()), (NAMES[i], slope, want)


@pytest.mark.parametrize("S", [4, 150])
def test_padding_may_hold_anything(S):
    note(f"hc_gated_delta_backward S={S}: NaN behind the lengths")
    ins = inputs(4, S, 1, 2, 40, 24, "bf16", seed=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    do = torch.randn(4, S, 2, 24, device="cuda", generator=g).bfloat16()
    dM = torch.randn(4, 2, 40, 24, device="cuda", generator=g)
    L = torch.tensor([S // 2, 0, S + 9, -3], dtype=torch.int32, device="cuda")
    want = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM, lengths=L)
    assert torch.equal(want[5][[1, 3]], dM[[1, 3]])
    for t in (*ins[:5], do):
        t[0, S // 2:] = float("nan")
        t[1], t[3] = float("nan"), float("nan")
    junk = [torch.full_like(t, 7) for t in want]
    got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM, lengths=L, out=junk)
    assert all(a is b for a, b in zip(got, junk))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t in got[:5]:
        assert not t[0, S // 2:].any() and not t[1].any() and not t[3].any()


def test_without_states_and_empty():
    note("hc_gated_delta_backward without states, S = 0, B = 0")
    ins = inputs(2, 100, 1, 2, 32, 32, "f32", seed=3)
    do, z = torch.randn(2, 100, 2, 32, device="cuda"), torch.zeros(2, 2, 32, 32, device="cuda")
    a = hc.hc_gated_delta_backward(*ins[:5], do)
    b = hc.hc_gated_delta_backward(*ins[:5], do, z, z)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    e = [t[:, :0].contiguous() for t in ins[:5]]
    assert torch.equal(hc.hc_gated_delta_backward(*e, do[:, :0].contiguous(), ins[5], ins[5])[5], ins[5])
    e = [t[:0].contiguous() for t in ins[:5]]
    assert hc.hc_gated_delta_backward(*e, do[:0].contiguous())[0].shape == (0, 100, 1, 32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decays_at_the_ends_of_their_range(dt):
    note(f"hc_gated_delta_backward decays of -inf, -1000 and 0 {dt}")
    ins = inputs(1, 140, 1, 1, 32, 32, dt, seed=5)
    rng = np.random.default_rng(6)
    do, dM = up(rng.normal(size=(1, 140, 1, 32)), dt), up(rng.normal(size=(1, 1, 32, 32)))
    for at, value in ((slice(70, 71), -1000.0), (slice(0, 71), -1000.0), (slice(0, 140), 0.0)):
        ins[3][:, at] = value
        got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM)
        torch.cuda.synchronize()
        check_backward(got, ins, do, dM, None, dt)
    ins[3][:, 70] = float("-inf")
    inf = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM)
    ins[3][:, 70] = -1000.0  # both are 0 in float32
    got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM)
    assert all(torch.equal(a, b) for a, b in zip(inf, got))


def test_beta_of_zero_and_one():
    note("hc_gated_delta_backward: beta 0 and 1")
    ins = inputs(1, 100, 1, 2, 64, 32, "f32", seed=6)
    ins[4][:, ::3], ins[4][:, 1::3] = 0, 1
    do, dM = torch.randn(1, 100, 2, 32, device="cuda"), torch.randn(1, 2, 64, 32, device="cuda")
    got = hc.hc_gated_delta_backward(*ins[:5], do, ins[5], dM, scale=0.7)
    torch.cuda.synchronize()
    check_backward(got, ins, do, dM, None, "f32", 0.7)
    assert not got[2][:, ::3].any() and got[4][:, ::3].any()


def test_unaligned_arrays():
    note("hc_gated_delta_backward on arrays one element off an aligned address")
    for dt in ("bf16", "f32"):
        ins = inputs(1, 100, 1, 2, 64, 64, dt, seed=8)
        ins.insert(5, torch.randn(1, 100, 2, 64, device="cuda").to(ins[0].dtype))

        def off(t):
            big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            big[1:] = t.reshape(-1)
            return big[1:].view(t.shape)

        a = hc.hc_gated_delta_backward(*ins)
        b = hc.hc_gated_delta_backward(*[off(t) for t in ins])
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_binding_refuses():
    q, k, v, g, be, M = inputs(2, 10, 1, 2, 16, 16, "f32")
    f = hc.hc_gated_delta_backward
    for bad in (lambda: f(q, k, v, g, be, v[:1]), lambda: f(q, k, v, g, be, v, M[:1]), lambda: f(q, k, v, g, be, v, M, M[:1]),
                lambda: f(q, k, v, g, be, v, out=(k[:1],) + (None,) * 5)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        f(q, k, v, g, be, v.bfloat16())
    with pytest.raises(hc.HCError):
        f(q, k, v, g, be, v, out=(q,) + (None,) * 5)
