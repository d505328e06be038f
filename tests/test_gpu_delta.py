"""The gated delta rule on the GPU against its float64 form (oracle/sublayer_ops.py).

Bounds are on norms, for each head. A product of operands in two bfloat16 parts is off by at most
3 x 2^-18 of its terms' magnitudes (2^-18 for what two parts leave of each factor, 2^-18 for the
two low parts' product), and its sum of at most 256 float32 roundings by 2^-16 more: c = 2^-15 in all.
With unit keys and 0 <= beta <= 1 a token's map of the state has no norm above 1, so that what a
chunk's products add to the state's error is not amplified by later ones; _bounds() adds it up
chunk by chunk from the magnitudes of the products' terms. Single tokens are plain float32 sums
and lie far within it. A bfloat16 output rounds by 2^-8 of each element.
"""
import numpy as np
import pytest

from hc_testutil import have_gpu, note
from oracle import sublayer_ops as R

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc

P = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
C15 = 2.0 ** -15


def up(a, dt="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to({"f32": torch.float32, "bf16": torch.bfloat16}[dt])


def down(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(B, S, Hk, Hv, Dk, Dv, dt, seed=0, decay=(-7, 0.5)):
    """q, k, v, g, beta, state on the device: unit keys, decays over a few to a thousand tokens."""
    rng = np.random.default_rng(seed)
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)  # noqa: E731
    return [up(unit(rng.normal(size=(B, S, Hk, Dk))), dt), up(unit(rng.normal(size=(B, S, Hk, Dk))), dt),
            up(rng.normal(size=(B, S, Hv, Dv)), dt), up(-np.exp(rng.uniform(*decay, size=(B, S, Hv)))),
            up(1 / (1 + np.exp(-rng.normal(size=(B, S, Hv))))), up(0.3 * rng.normal(size=(B, Hv, Dk, Dv)))]


def _norm(a):
    return np.linalg.norm(a)  # Frobenius


def _two(a):
    return np.linalg.norm(a, 2)


def _bounds(q, k, v, g, beta, M, scale, n):
    """(bound on the norm of o's error, of the state's) of one head's n tokens; unit keys."""
    eo2, em = 0.0, 0.0
    for t in range(0, n, 64):
        Q, K, V, G, b = q[t:t + 64][:n - t], k[t:t + 64][:n - t], v[t:t + 64][:n - t], g[t:t + 64][:n - t], beta[t:t + 64][:n - t]
        Gs = np.cumsum(G)
        D = np.tril(np.exp(np.minimum(Gs[:, None] - Gs[None], 0)))
        A, Pm = np.tril(D * (K @ K.T), -1) * b, D * (Q @ K.T)
        T = np.linalg.inv(np.eye(len(G)) + A)
        ahead, end = np.exp(Gs)[:, None], np.exp(Gs[-1] - Gs)[:, None]
        r = V - ahead * (K @ M)
        x = b[:, None] * (T @ r)
        ab = np.abs
        er = C15 * _norm(ab(V) + ahead * (ab(K) @ ab(M)))
        ez = _two(T) * er + C15 * _norm(ab(T) @ (np.eye(len(G)) + ab(A)) @ ab(T) @ ab(r)) + C15 * _norm(ab(T) @ ab(r))
        ex = b.max() * ez + C15 * _norm(x)
        new = _two(K * end) * ex + C15 * _norm(ab(M) + ab(K * end).T @ ab(x))
        o = scale * (_norm(Q) * em + _two(Pm) * ex + C15 * _norm(ahead * (ab(Q) @ ab(M)) + 2 * ab(Pm) @ ab(x)))
        eo2 += o * o
        em += new
        M = np.exp(Gs[-1]) * M + (K * end).T @ x
    return np.sqrt(eo2), em


def check_forward(got_o, got_M, ins, lengths, dt, scale=None, o_init=None, slack=1):
    q, k, v, g, beta, M = (down(x) for x in ins)
    B, S, Hk, Dk = q.shape
    Hv = v.shape[2]
    scale = Dk ** -0.5 if scale is None else scale
    ro, rM = R.gated_delta(q, k, v, g, beta, M, lengths, scale, o_init)
    o, Mg = down(got_o), down(got_M)
    for b in range(B):
        n = S if lengths is None else int(np.clip(lengths[b], 0, S))
        for h in range(Hv):
            kh = h // (Hv // Hk)
            eo, em = _bounds(q[b, :, kh], k[b, :, kh], v[b, :, h], g[b, :, h], beta[b, :, h], M[b, h], scale, n)
            eo, em = slack * eo, slack * em
            err = np.abs(o[b, :n, h] - ro[b, :n, h])
            # what is not the rounding of the element itself
            more = np.maximum(err - P[dt] * (np.abs(ro[b, :n, h]) + err), 0)
            assert np.isfinite(o[b, :n, h]).all() and _norm(more) <= eo, (b, h, _norm(more), eo)
            assert np.isfinite(Mg[b, h]).all() and _norm(Mg[b, h] - rM[b, h]) <= em + 2.0 ** -22 * _norm(rM[b, h]), \
                (b, h, _norm(Mg[b, h] - rM[b, h]), em)
            if o_init is not None:
                assert np.array_equal(o[b, n:, h], o_init[b, n:, h]), "rows behind the length changed"


# B, S, Hk, Hv, Dk, Dv: one token, around a chunk, several; odd sizes; every width's variants
SIZES = [(1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 128, 128), (2, 5, 1, 3, 100, 36), (1, 8, 1, 1, 256, 256), (2, 9, 1, 1, 64, 64),
         (1, 63, 1, 2, 24, 40), (2, 64, 2, 2, 128, 64), (1, 65, 1, 1, 128, 128), (2, 200, 1, 3, 72, 100),
         (1, 129, 1, 1, 200, 30), (1, 192, 1, 1, 256, 256), (1, 70, 2, 2, 33, 17), (1, 130, 1, 1, 7, 130),
         (1, 100, 1, 1, 129, 66), (1, 1000, 1, 1, 64, 128)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward(size, dt):
    B, S, Hk, Hv, Dk, Dv = size
    rng = np.random.default_rng(S)
    ins = inputs(*size, dt, seed=S + Dk)
    for L in (None, rng.integers(0, S + 1, size=B)):
        note(f"hc_gated_delta {size} {dt} lengths={L}")
        o0 = up(rng.normal(size=(B, S, Hv, Dv)), dt)
        lengths = None if L is None else torch.from_numpy(L.astype(np.int32)).cuda()
        o, M = hc.hc_gated_delta(*ins, lengths=lengths, out=(o0.clone(), None))
        torch.cuda.synchronize()
        check_forward(o, M, ins, L, dt, o_init=down(o0))


@pytest.mark.parametrize("size", [(3, 1500, 1, 1, 64, 24), (2, 1024, 1, 2, 40, 80), (1, 1100, 1, 1, 130, 66)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_segments(size, dt):
    """Few heads and long sequences are walked in segments that are joined afterwards: lengths that end in
    the first, at a border, in the middle and in the last of them. The segments' maps are products of the
    same kind, off by the same c of terms whose norms are at most 1: twice the chunks' bounds."""
    B, S, Hk, Hv, Dk, Dv = size
    ins = inputs(*size, dt, seed=S)
    rng = np.random.default_rng(S)
    ends = [S, 256, 0, 257, 700, 1, 512, S - 1]
    for turn in range(0, len(ends), B):
        L = np.array((ends[turn:] + ends)[:B])
        note(f"hc_gated_delta {size} {dt} lengths={L}")
        o0 = up(rng.normal(size=(B, S, Hv, Dv)), dt)
        o, M = hc.hc_gated_delta(*ins, lengths=torch.from_numpy(L.astype(np.int32)).cuda(), out=(o0.clone(), None))
        torch.cuda.synchronize()
        check_forward(o, M, ins, L, dt, o_init=down(o0), slack=2)


@pytest.mark.parametrize("S", [4, 150])
def test_padding_may_hold_anything(S):
    note(f"hc_gated_delta S={S}: NaN behind the lengths, lengths out of range")
    ins = inputs(4, S, 1, 2, 40, 24, "bf16", seed=1)
    L = torch.tensor([S // 2, 0, S + 9, -3], dtype=torch.int32, device="cuda")
    want, wantM = hc.hc_gated_delta(*ins, lengths=L)
    assert not want[1].any() and not want[3].any() and not want[0, S // 2:].any()
    assert torch.equal(wantM[[1, 3]], ins[5][[1, 3]])
    for t in ins[:5]:
        t[0, S // 2:] = float("nan")
        t[1], t[3] = float("nan"), float("nan")
    o, M = hc.hc_gated_delta(*ins, lengths=L)
    assert torch.equal(o, want) and torch.equal(M, wantM)
    alone = hc.hc_gated_delta(*[t[2:3].contiguous() for t in ins])
    assert torch.equal(o[2:3], alone[0]) and torch.equal(M[2:3], alone[1])


@pytest.mark.parametrize("S", [3, 200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shared_heads_are_repeated_heads(S, dt):
    note(f"hc_gated_delta S={S} {dt}: shared key heads")
    q, k, v, g, be, M = inputs(2, S, 2, 6, 64, 48, dt, seed=2)
    o, last = hc.hc_gated_delta(q, k, v, g, be, M)
    rep = lambda t: t.repeat_interleave(3, 2).contiguous()  # noqa: E731
    o2, last2 = hc.hc_gated_delta(rep(q), rep(k), v, g, be, M)
    assert torch.equal(o, o2) and torch.equal(last, last2)


def test_without_states_and_empty():
    note("hc_gated_delta without states, S = 0, B = 0")
    for S in (5, 100):
        q, k, v, g, be, M = inputs(2, S, 1, 2, 32, 32, "f32")
        o, last = hc.hc_gated_delta(q, k, v, g, be)
        o2, last2 = hc.hc_gated_delta(q, k, v, g, be, torch.zeros_like(M))
        assert torch.equal(o, o2) and torch.equal(last, last2)
        assert hc.hc_gated_delta(q, k, v, g, be, want_state=False)[1] is None
    e = [t[:, :0].contiguous() for t in (q, k, v, g, be)]
    o, last = hc.hc_gated_delta(*e, M)
    assert o.shape == (2, 0, 2, 32) and torch.equal(last, M)
    assert not hc.hc_gated_delta(*e)[1].any()
    e = [t[:0].contiguous() for t in (q, k, v, g, be)]
    assert hc.hc_gated_delta(*e)[0].shape == (0, 100, 2, 32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_goes_on_from_its_state(dt):
    """In pieces of one token, a few and chunks, the state in place: the bounds of the whole, once more for
    the other order of the same products."""
    note(f"hc_gated_delta in pieces {dt}")
    ins = inputs(2, 300, 1, 2, 72, 40, dt, seed=4)
    state, parts = ins[5].clone(), []
    for t0, t1 in ((0, 1), (1, 6), (6, 100), (100, 228), (228, 229), (229, 300)):
        o, s = hc.hc_gated_delta(*[t[:, t0:t1].contiguous() for t in ins[:5]], state, out=(None, state))
        assert s is state
        parts.append(o)
    torch.cuda.synchronize()
    check_forward(torch.cat(parts, 1), state, ins, None, dt)


@pytest.mark.parametrize("S", [4, 150])
def test_decays_at_the_ends_of_their_range(S):
    """-inf forgets: what follows is what a sequence that starts there gives; 0 keeps; long sums of strong
    decays leave their neighbours' differences alone."""
    note(f"hc_gated_delta S={S}: decays of -inf, 0 and -1000")
    q, k, v, g, be, M = inputs(1, S, 1, 1, 32, 32, "f32", seed=5)
    cut = S // 2
    g[:, cut] = float("-inf")
    o, last = hc.hc_gated_delta(q, k, v, g, be, M)
    tail = [t[:, cut:].contiguous() for t in (q, k, v, g, be)]
    tail[3][:, 0] = 0
    o2, last2 = hc.hc_gated_delta(*tail)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all()
    fresh = [q[:, cut:], k[:, cut:], v[:, cut:], tail[3], be[:, cut:], torch.zeros_like(M)]
    check_forward(o[:, cut:].contiguous(), last, fresh, None, "f32")
    check_forward(o2, last2, fresh, None, "f32")
    g[:, :cut + 1] = -1000
    g[:, cut + 1:] = -0.01
    o, last = hc.hc_gated_delta(q, k, v, g, be, M)
    torch.cuda.synchronize()
    check_forward(o, last, [q, k, v, g, be, M], None, "f32")
    g[:] = 0
    o, last = hc.hc_gated_delta(q, k, v, g, be, M)
    torch.cuda.synchronize()
    check_forward(o, last, [q, k, v, g, be, M], None, "f32")


def test_beta_of_zero_one_and_scale():
    note("hc_gated_delta: beta 0 and 1, scales")
    q, k, v, g, be, M = inputs(1, 100, 1, 1, 64, 32, "f32", seed=6)
    be[:, ::3], be[:, 1::3] = 0, 1
    for scale in (1.0, -0.5, 0.0):
        o, last = hc.hc_gated_delta(q, k, v, g, be, M, scale=scale)
        torch.cuda.synchronize()
        check_forward(o, last, [q, k, v, g, be, M], None, "f32", scale)


@pytest.mark.parametrize("S", [6, 7, 200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_beta_up_to_two(S, dt):
    """Up to beta = 2 a token's map of the state has no norm above 1 (but for bfloat16's rounding of unit keys,
    2 x 2 x 2^-9 of it a token at most, e^(S 2^-7) over all of them). Six tokens go one by one, seven as a chunk."""
    note(f"beta in (0, 2), S={S}")
    ins = inputs(2, S, 1, 2, 64, 40, dt, seed=77)
    ins[4] = 2 * ins[4]
    o, M = hc.hc_gated_delta(*ins)
    check_forward(o, M, ins, None, dt, slack=np.exp(S * 2.0 ** -7) if dt == "bf16" else 1)


@pytest.mark.parametrize("S", [2, 90])
def test_a_nan_stays_in_its_head_and_later_tokens(S):
    note(f"hc_gated_delta S={S}: NaN")
    ins = inputs(2, S, 2, 2, 32, 32, "f32", seed=7)
    want, wantM = hc.hc_gated_delta(*ins)
    ins[2][0, S - 1, 1, 3] = float("nan")
    o, M = hc.hc_gated_delta(*ins)
    assert torch.equal(o[1], want[1]) and torch.equal(o[0, :, 0], want[0, :, 0]) and torch.equal(M[1], wantM[1])
    assert o[0, S - 1, 1, 3].isnan() and M[0, 1, :, 3].isnan().all() and not M[0, 1, :, 4:].isnan().any()


def test_unaligned_arrays():
    note("hc_gated_delta on arrays one element off an aligned address")
    for S in (3, 100):
        for dt in ("bf16", "f32"):
            ins = inputs(1, S, 1, 2, 64, 64, dt, seed=8)

            def off(t):
                big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
                big[1:] = t.reshape(-1)
                return big[1:].view(t.shape)

            o, M = hc.hc_gated_delta(*ins)
            o2, M2 = hc.hc_gated_delta(*[off(t) for t in ins])
            assert torch.equal(o, o2) and torch.equal(M, M2)


def test_binding_refuses():
    q, k, v, g, be, M = inputs(2, 10, 1, 2, 16, 16, "f32")
    f = hc.hc_gated_delta
    for bad in (lambda: f(q[0], k, v, g, be), lambda: f(q, k[:, :5], v, g, be), lambda: f(q, k, v[0], g, be),
                lambda: f(q, k, v[:, :5].contiguous(), g, be), lambda: f(q, k, v, g[..., :1].contiguous(), be),
                lambda: f(q, k, v, g, be, M[:1]), lambda: f(q.transpose(1, 2), k, v, g, be),
                lambda: f(q.repeat(1, 1, 3, 1), k.repeat(1, 1, 3, 1), v, g, be),
                lambda: f(q, k, v, g, be, lengths=torch.ones(3, dtype=torch.int32, device="cuda")),
                lambda: f(q, k, v, g, be, out=(v[:1], None)), lambda: f(q, k, v, g, be, out=(None, M[:1]))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(q.half(), k, v, g, be), lambda: f(q, k.bfloat16(), v, g, be), lambda: f(q, k, v, g.double(), be),
                lambda: f(q.cpu(), k, v, g, be), lambda: f(q, k, v, g, be, M.bfloat16()),
                lambda: f(q, k, v, g, be, lengths=torch.ones(2, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    big = torch.zeros(1, 1, 1, 257, device="cuda")
    with pytest.raises((ValueError, hc.HCError)):
        f(big, big, big[..., :1].contiguous(), big[..., 0].contiguous(), big[..., 0].contiguous())
    with pytest.raises(hc.HCError):
        f(q, k, v, g, be, out=(v, None))
