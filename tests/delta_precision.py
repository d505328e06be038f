"""What the tests of the gated delta rule's precision share: inputs, tolerances, and the chunked form in
float64 with mistakes to plant in it (tests/test_delta_precision.py shows that the tolerances tell them).

Tolerances are on the norm of a head's error, relative to the norm of the result. Every factor of a
product keeps 24 bits, so what remains are the roundings of float32 sums, 2^-24 of what is summed each:
a sum of n terms of random signs is off by sqrt(n) 2^-24 of its norm.
  State: what a chunk adds is a sum over 64 tokens, sqrt(64) 2^-24 = 2^-21.
  Outputs and gradients: sums over up to 256 keys or columns, 2^-20 (the first state's too: what a chunk adds to it
  holds W, which is such a sum).
  dg: a sum over a chunk that two running sums of 64 pass through one after the other: 2^-19.
  A bfloat16 result against the float64 one rounded to bfloat16, half(): off by e of its rms before it is
  rounded, an element that is u steps of its type, u from 2^-8 to 2^-7 of it, falls on the other side of a
  rounding for one in e / u and is then u off: sqrt(e u) of the norm, 2^-14 for e = 2^-20. The N 2^-12.5
  elements that do so are counted like dice, three times their spread on top, and where N is small
  one of them may be the largest of all.
  Sequences in segments, joins(): one of 256 tokens and more hands its state to the next by one more such product,
  whose errors stay where the state does: as many of them as there are segments, of random signs.
"""
import numpy as np

STATE, OUT, DG = 2.0 ** -21, 2.0 ** -20, 2.0 ** -19


def half(y):
    """The tolerance of a bfloat16 result whose rounded float64 form is y."""
    tol = 2.0 ** -14 * np.sqrt(1 + 6 / np.sqrt(y.size * 2.0 ** -12.5))
    return tol if y.size >= 1 << 18 else tol + 2.0 ** -7 * np.abs(y).max() / np.linalg.norm(y)


def joins(S):
    """What the tolerances grow by where S tokens are walked in segments."""
    return max(1.0, np.sqrt(S / 256))


def bf16(a):
    """Rounded to bfloat16, ties to even."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)


def inputs(B, S, Hk, Hv, Dk, Dv, dt, seed, slow=None):
    """q, k, v, g, beta, state, do, dstate as float64 arrays of float32 or bfloat16 values. Heads forget over a few to a
    thousand tokens, as the measured cases do; with `slow` every token keeps all but about that share and writes
    little, so that the first state reaches the last."""
    rng = np.random.default_rng(seed)
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)  # noqa: E731
    stream = bf16 if dt == "bf16" else (lambda a: a.astype(np.float32).astype(np.float64))
    f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    q, k = unit(rng.normal(size=(B, S, Hk, Dk))), unit(rng.normal(size=(B, S, Hk, Dk)))
    g = -np.exp(-1 - 6 * rng.uniform(size=Hv)) * rng.uniform(0.2, 2.2, size=(B, S, Hv))
    beta = 1 / (1 + np.exp(-rng.normal(size=(B, S, Hv))))
    if slow is not None:
        g, beta = -slow * rng.uniform(0.2, 2, size=(B, S, Hv)), rng.uniform(0.002, 0.01, size=(B, S, Hv))
    return [stream(q), stream(k), stream(rng.normal(size=(B, S, Hv, Dv))), f32(g), f32(beta),
            f32(0.3 * rng.normal(size=(B, Hv, Dk, Dv))), stream(0.1 * rng.normal(size=(B, S, Hv, Dv))),
            f32(0.1 * rng.normal(size=(B, Hv, Dk, Dv)))]


def rel(x, y):
    return np.linalg.norm(np.asarray(x, np.float64) - y) / np.linalg.norm(y)


def parts(x, n):
    """x as the sum of n bfloat16 values (None: as it is)."""
    if n is None:
        return x
    got = np.zeros_like(x)
    for _ in range(n):
        got = got + bf16(x - got)
    return got


def chunked(q, k, v, g, beta, M, scale, held=None, segment=None, maps=None, map_parts=None):
    """(o, last state) of one head in chunks of 64. held: parts in which a product's factors are kept; segment:
    tokens of a segment that is walked from zeros and joined by its map; maps "zero": by none; map_parts: parts of
    the map and of the state that it is applied to."""
    P = lambda x: parts(x, held)  # noqa: E731
    Dk, out = q.shape[1], []

    def walk(lo, hi, M, keys_only=False, keep=None):
        for t in range(lo, hi, 64):
            at = slice(t, min(hi, t + 64))
            Q, K, V, G, b = q[at], k[at], v[at], np.cumsum(g[at]), beta[at][:, None]
            if keys_only:
                V = np.zeros((len(Q), M.shape[1]))
            D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
            T = np.linalg.inv(np.eye(len(G)) + np.tril(D * (P(K) @ P(K).T), -1) * b.T)
            Pm, ahead, end = D * (P(Q) @ P(K).T), np.exp(G)[:, None], np.exp(G[-1] - G)[:, None]
            x = b * (P(T) @ P(V - ahead * (P(K) @ P(M))))
            if keep is not None:
                keep.append(scale * (ahead * (P(Q) @ P(M)) + P(Pm) @ P(x)))
            M = np.exp(G[-1]) * M + P(K).T @ P(end * x)
        return M

    n = len(q)
    if segment is None:
        return (lambda last: (np.concatenate(out), last))(walk(0, n, M, keep=out))
    state = M
    for lo in range(0, n, segment):
        hi = min(n, lo + segment)
        start, zeros = state, np.zeros_like(M)
        last = walk(lo, hi, start, keep=out)
        if lo == 0 or hi == n:
            state = last
        else:
            Phi = walk(lo, hi, np.eye(Dk), keys_only=True) if maps != "zero" else np.zeros((Dk, Dk))
            state = walk(lo, hi, zeros) + parts(Phi, map_parts) @ parts(state, map_parts)
    return np.concatenate(out), last


def dg_size(ins, n, b, h):
    """The norm over n tokens of ||F|| ||dF|| / sqrt(Dk Dv) of one head, the size of dg = <dF, F> of unrelated states.
    Where both hardly change from token to token the sum of one token's products cancels as that of all others
    does, and dg can be small beside it. An error e of the states' elements, relative to their rms and of random
    signs, is e ||F|| ||dF|| / sqrt(Dk Dv) in the sum of products, whatever the sum itself comes to."""
    q, k, v, g, beta, M, do, dM = ins
    kh = h // (v.shape[2] // k.shape[2])
    m, r, scale, F = M[b, h], dM[b, h], q.shape[3] ** -0.5, []
    for t in range(n):
        F.append(np.exp(g[b, t, h]) * m)
        kt = k[b, t, kh]
        m = F[-1] + beta[b, t, h] * np.outer(kt, v[b, t, h] - F[-1].T @ kt)
    size = 0.0
    for t in range(n - 1, -1, -1):
        kt = k[b, t, kh]
        r = r + np.outer(q[b, t, kh], scale * do[b, t, h])
        dF = r - np.outer(kt, beta[b, t, h] * (r.T @ kt))
        size += np.sum(F[t] ** 2) * np.sum(dF ** 2) / m.size
        r = np.exp(g[b, t, h]) * dF
    return np.sqrt(size)
