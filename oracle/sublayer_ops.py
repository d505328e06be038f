"""Plain float64 forms of the operators beside the stream mixing (tests only).

The root-mean-square norm and the layer norm with their 8-bit codes, the gated linear
recurrence, the router's balance loss and the router's backward, each with its gradient,
written one token at a time from the definitions in include/hc.h.
"""
from __future__ import annotations

import numpy as np

QMAX = {"e4m3": 448.0, "i8": 127.0}


def sigmoid(z):
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


# -------------------------------------------------------------------- norm


def rms_norm(v, weight, eps):
    """y of rows v [T, C]; a row whose mean square + eps is 0 gives 0."""
    v = np.asarray(v, np.float64)
    w = np.ones(v.shape[1]) if weight is None else np.asarray(weight, np.float64)
    ms = (v * v).mean(1, keepdims=True) + eps
    rstd = np.where(ms > 0, 1 / np.sqrt(np.where(ms > 0, ms, 1)), 0.0)
    return v * rstd * w


def rms_norm_backward(v, weight, eps, dy, ds=None):
    """(dx, dweight)."""
    v, dy = np.asarray(v, np.float64), np.asarray(dy, np.float64)
    w = np.ones(v.shape[1]) if weight is None else np.asarray(weight, np.float64)
    ms = (v * v).mean(1, keepdims=True) + eps
    rstd = np.where(ms > 0, 1 / np.sqrt(np.where(ms > 0, ms, 1)), 0.0)
    vh = v * rstd
    dx = rstd * (w * dy - vh * (w * dy * vh).mean(1, keepdims=True))
    if ds is not None:
        dx = dx + np.asarray(ds, np.float64)
    return dx, (dy * vh).sum(0)


def layer_norm(v, weight, bias, eps):
    """y of rows v [T, C]; a row whose variance + eps is 0 gives the bias."""
    v = np.asarray(v, np.float64)
    w = np.ones(v.shape[1]) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(v.shape[1]) if bias is None else np.asarray(bias, np.float64)
    d = v - v.mean(1, keepdims=True)
    var = (d * d).mean(1, keepdims=True) + eps
    rstd = np.where(var > 0, 1 / np.sqrt(np.where(var > 0, var, 1)), 0.0)
    return d * rstd * w + b


def layer_norm_backward(v, weight, eps, dy, ds=None):
    """(dx, dweight, dbias)."""
    v, dy = np.asarray(v, np.float64), np.asarray(dy, np.float64)
    w = np.ones(v.shape[1]) if weight is None else np.asarray(weight, np.float64)
    d = v - v.mean(1, keepdims=True)
    var = (d * d).mean(1, keepdims=True) + eps
    rstd = np.where(var > 0, 1 / np.sqrt(np.where(var > 0, var, 1)), 0.0)
    n, u = d * rstd, w * dy
    dx = rstd * (u - u.mean(1, keepdims=True) - n * (u * n).mean(1, keepdims=True))
    if ds is not None:
        dx = dx + np.asarray(ds, np.float64)
    return dx, (dy * n).sum(0), dy.sum(0)


def quant_scales(y, kind, group):
    """scale [T, groups] of y [T, C]."""
    T, C = y.shape
    width = group or C
    cols = [np.abs(y[:, c:c + width]).max(1) / QMAX[kind] for c in range(0, C, width)]
    scale = np.stack(cols, 1)
    return np.where(scale < 2.0 ** -126, 1.0, scale)


def per_channel(scale, C, group):
    """scale [T, groups] spread over the channels, [T, C]."""
    return np.repeat(scale, group or C, axis=1)[:, :C]


# --------------------------------------------------------------------- scan


def gated_scan(x, gate, h0=None, lengths=None, tied=True, y_init=None):
    """(y [B, S, C], h_last [B, C]); rows behind a length keep y_init."""
    x, gate = np.asarray(x, np.float64), np.asarray(gate, np.float64)
    B, S, C = x.shape
    a = sigmoid(gate)
    u = sigmoid(-gate) if tied else np.ones_like(a)
    y = np.zeros((B, S, C)) if y_init is None else np.array(y_init, np.float64)
    h = np.zeros((B, C)) if h0 is None else np.array(h0, np.float64)
    for b in range(B):
        n = S if lengths is None else int(np.clip(lengths[b], 0, S))
        for t in range(n):
            h[b] = a[b, t] * h[b] + u[b, t] * x[b, t]
            y[b, t] = h[b]
    return y, h


def gated_scan_backward(x, gate, y, dy, h0=None, dh_last=None, lengths=None, tied=True):
    """(dx, dgate, dh0) with h_{t-1} taken from y."""
    x, gate, y, dy = (np.asarray(v, np.float64) for v in (x, gate, y, dy))
    B, S, C = x.shape
    a, u = sigmoid(gate), sigmoid(-gate)
    R = np.zeros((B, C)) if dh_last is None else np.array(dh_last, np.float64)
    first = np.zeros((B, C)) if h0 is None else np.asarray(h0, np.float64)
    dx, dgate = np.zeros((B, S, C)), np.zeros((B, S, C))
    for b in range(B):
        n = S if lengths is None else int(np.clip(lengths[b], 0, S))
        for t in range(n - 1, -1, -1):
            dh = dy[b, t] + R[b]
            prev = y[b, t - 1] if t else first[b]
            dx[b, t] = (u[b, t] if tied else 1.0) * dh
            dgate[b, t] = dh * (prev - x[b, t] if tied else prev) * a[b, t] * u[b, t]
            R[b] = a[b, t] * dh
    return dx, dgate, R


# --------------------------------------------------------------- delta rule


def gated_delta(q, k, v, g, beta, state=None, lengths=None, scale=None, o_init=None):
    """(o [B, S, Hv, Dv], last state [B, Hv, Dk, Dv]); rows behind a length keep o_init."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    B, S, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    scale = Dk ** -0.5 if scale is None else scale
    o = np.zeros((B, S, Hv, Dv)) if o_init is None else np.array(o_init, np.float64)
    M = np.zeros((B, Hv, Dk, Dv)) if state is None else np.array(state, np.float64)
    for b in range(B):
        n = S if lengths is None else int(np.clip(lengths[b], 0, S))
        for h in range(Hv):
            m, kh = M[b, h], h // (Hv // Hk)
            for t in range(n):
                kt = k[b, t, kh]
                F = np.exp(g[b, t, h]) * m
                m = F + beta[b, t, h] * np.outer(kt, v[b, t, h] - F.T @ kt)
                o[b, t, h] = scale * (m.T @ q[b, t, kh])
            M[b, h] = m
    return o, M


def gated_delta_backward(q, k, v, g, beta, do, state=None, dstate=None, lengths=None, scale=None):
    """(dq, dk, dv, dg, dbeta, dstate0)."""
    q, k, v, g, beta, do = (np.asarray(x, np.float64) for x in (q, k, v, g, beta, do))
    B, S, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    scale = Dk ** -0.5 if scale is None else scale
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    R = np.zeros((B, Hv, Dk, Dv)) if dstate is None else np.array(dstate, np.float64)
    for b in range(B):
        n = S if lengths is None else int(np.clip(lengths[b], 0, S))
        for h in range(Hv):
            kh = h // (Hv // Hk)
            m = np.zeros((Dk, Dv)) if state is None else np.asarray(state[b, h], np.float64)
            steps = []
            for t in range(n):
                kt = k[b, t, kh]
                F = np.exp(g[b, t, h]) * m
                z = v[b, t, h] - F.T @ kt
                m = F + beta[b, t, h] * np.outer(kt, z)
                steps.append((F, z, m))
            r = R[b, h]
            for t in range(n - 1, -1, -1):
                F, z, m = steps[t]
                kt = k[b, t, kh]
                d = scale * do[b, t, h]
                r = r + np.outer(q[b, t, kh], d)
                dz = beta[b, t, h] * (r.T @ kt)
                dF = r - np.outer(kt, dz)
                dq[b, t, kh] += m @ d
                dk[b, t, kh] += beta[b, t, h] * (r @ z) - F @ dz
                dv[b, t, h] = dz
                db[b, t, h] = (r.T @ kt) @ z
                dg[b, t, h] = (dF * F).sum()
                r = np.exp(g[b, t, h]) * dF
            R[b, h] = r
    return dq, dk, dv, dg, db, R


# ------------------------------------------------------------------- router


def balance_loss(score, idx, B, S, N, m, coef=1.0, mask=None):
    """dict(loss, count [B, N], tokens [B], mean_p [B, E])."""
    E, k = N - m, idx.shape[1]
    count, tokens = np.zeros((B, N), np.int64), np.zeros(B, np.int64)
    mean_p, loss = np.zeros((B, E)), 0.0
    for b in range(B):
        for t in range(b * S, b * S + S):
            if mask is not None and not mask[t]:
                continue
            tokens[b] += 1
            for i in idx[t]:
                if 0 <= i < N:
                    count[b, i] += 1
            s = np.asarray(score[t], np.float64)
            if s.sum() != 0:
                mean_p[b] += s / s.sum()
        n = max(1, tokens[b])
        mean_p[b] /= n
        loss += (count[b, m:] * E / ((k - m) * n) * mean_p[b]).sum()
    return dict(loss=coef * loss / B if B else 0.0, count=count, tokens=tokens, mean_p=mean_p)


def balance_loss_backward(score, count, tokens, k, B, S, N, m, coef=1.0, dloss=1.0, mask=None):
    E = N - m
    dscore = np.zeros((B * S, E))
    for t in range(B * S):
        if mask is not None and not mask[t]:
            continue
        b = t // S
        n = max(1, tokens[b])
        f = count[b, m:] * E / ((k - m) * n)
        s = np.asarray(score[t], np.float64)
        if s.sum() != 0:
            dscore[t] = dloss * coef / (B * n) * (f - (f * s).sum() / s.sum()) / s.sum()
    return dscore


def router_backward(X, w_router, score, dscore, dX):
    """(dX + the router's part [T, N, C], dw_router [NC, E])."""
    T, N, C = X.shape
    out = np.array(dX, np.float64)
    w = np.asarray(w_router, np.float64)
    dw = np.zeros_like(w)
    for t in range(T):
        d = np.asarray(dscore[t], np.float64)
        if not np.any(d != 0):
            continue
        x = np.asarray(X[t], np.float64).reshape(-1)
        r2 = (x * x).mean()
        if r2 == 0:
            continue
        s = np.asarray(score[t], np.float64)
        dz = d * s * (1 - s)
        inside = dz != 0
        z = np.log(s[inside]) - np.log1p(-s[inside])
        out[t] += (w @ dz / np.sqrt(r2) - x * (dz[inside] * z).sum() / (r2 * N * C)).reshape(N, C)
        dw += np.outer(x, dz / np.sqrt(r2))
    return out, dw
