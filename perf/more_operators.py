"""The layer norm and the gated delta rule, as measurable cases.

Two operators of hc.h, each with its gradient: the layer norm in front of a
sublayer function (with the residual's addition or the pre-read of the streams),
and the gated delta rule inside it, the linear recurrence whose state is a matrix
per head, over whole sequences or token by token.

run() computes a case's operator once: in plain float32 torch operations, or with
`own` set through the package. exact() is the definition in float64.
"""
import math

import torch

own = False

F8_MAX = 448.0  # largest finite e4m3
TINY = 2.0 ** -126  # smallest normal float32: a smaller scale is replaced by 1
CHUNK = 64  # tokens that the plain form of the delta rule joins at once
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # serving, one decode step of 16 requests: the residual joins, latency counts
        dict(name="ln_decode", op="norm", T=16, C=4096, dtype="bf16", quant="", group=0),
        # a prefill chunk whose projections read 8 bits, a scale for each 128 channels
        dict(name="ln_prefill", op="norm", T=8192, C=4096, dtype="bf16", quant="e4m3", group=128),
        # training forward: pre-read of 4 streams and norm in one pass, F_in kept for the backward
        dict(name="pre_ln_train", op="pre_norm", T=8192, n=4, C=4096, dtype="bf16", quant="", group=0),
        # its backward, with the residual's own gradient joined, an odd number of tokens
        dict(name="ln_backward", op="norm_backward", T=8191, C=4096, dtype="bf16"),
        # a small model in float32, odd sizes
        dict(name="ln_backward_odd", op="norm_backward", T=1021, C=1100, dtype="f32"),
        # serving, one new token of one request: latency counts
        dict(name="delta_step_one", op="delta", B=1, S=1, Hk=16, Hv=16, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # serving, one new token for each of 64 requests, two value heads to a key head
        dict(name="delta_step", op="delta", B=64, S=1, Hk=16, Hv=32, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # one long prompt: few heads, a long way through them
        dict(name="delta_long", op="delta", B=1, S=8192, Hk=16, Hv=16, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # training forward of a batch with shared key heads
        dict(name="delta_batch", op="delta", B=8, S=1024, Hk=8, Hv=16, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a padded batch in float32, odd sizes
        dict(name="delta_padded", op="delta", B=5, S=509, Hk=3, Hv=6, Dk=72, Dv=100, dtype="f32", ragged=True),
        # training backward of two sequences
        dict(name="delta_backward", op="delta_backward", B=2, S=4096, Hk=8, Hv=16, Dk=128, Dv=128, dtype="bf16",
             ragged=False),
        # the backward of a small padded batch
        dict(name="delta_backward_padded", op="delta_backward", B=3, S=333, Hk=4, Hv=4, Dk=64, Dv=128, dtype="bf16",
             ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pre_norm", "norm_backward", "delta", "delta", "delta", "delta_backward",
                     "delta_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "pre_norm"):
        quant = rng.choice(["", "e4m3"])
        c = dict(op=op, T=_log(rng, 1, 8192), C=_log(rng, 64, 8192), dtype=dtype, quant=quant,
                 group=rng.choice([0, 32, 64, 128]) if quant else 0)
        if rng.random() < 0.6:
            c["C"] = max(128, c["C"] // 128 * 128)
        if op == "pre_norm":
            c.update(n=rng.choice([2, 4, 4, 8]), T=_log(rng, 1, 2048))
        return c
    if op == "norm_backward":
        C = _log(rng, 64, 8192)
        return dict(op=op, T=_log(rng, 1, 8192), C=max(128, C // 128 * 128) if rng.random() < 0.6 else C, dtype=dtype)
    Hk, times = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3])
    if rng.random() < 0.7:
        Dk, Dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    else:
        Dk, Dv = _log(rng, 16, 256), _log(rng, 16, 256)
    most = (1 << 30) // (Hk * times * Dk * Dv)  # tokens
    B = _log(rng, 1, min(64, max(1, most)))
    S = _log(rng, 1, min(8192, max(1, most // B)))
    return dict(op=op, B=B, S=S, Hk=Hk, Hv=Hk * times, Dk=Dk, Dv=Dv, dtype=dtype, ragged=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)
    rn = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    uni = lambda *s: torch.rand(*s, device=dev, generator=g)  # noqa: E731
    op, dt, s = case["op"], DT[case["dtype"]], {"case": case}
    if op in ("norm", "pre_norm", "norm_backward"):
        T, C = case["T"], case["C"]
        s["weight"], s["bias"] = 1 + 0.2 * rn(C), 0.2 * rn(C)
        if op == "norm":
            # a residual stream grows over the layers, some channels far beyond the others and off centre
            size = torch.exp(0.7 * rn(C))
            s["residual"] = (4 * (rn(T, C) + 0.3 * rn(C)) * size).to(dt)
            s["x"] = rn(T, C).to(dt)
        elif op == "pre_norm":
            s["X"] = torch.empty(T, case["n"], C, dtype=dt, device=dev).normal_(generator=g)
            s["h_pre"] = torch.sigmoid(rn(T, case["n"]))
        else:
            s["s"] = (2 * rn(T, C) + 0.5).to(dt)
            s["dy"] = (0.1 * rn(T, C)).to(dt)
            s["ds"] = (0.1 * rn(T, C)).to(dt)
        return s
    B, S, Hk, Hv, Dk, Dv = (case[v] for v in ("B", "S", "Hk", "Hv", "Dk", "Dv"))
    unit = lambda t: t / t.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    s["q"], s["k"] = unit(rn(B, S, Hk, Dk)).to(dt), unit(rn(B, S, Hk, Dk)).to(dt)
    s["v"] = rn(B, S, Hv, Dv).to(dt)
    # heads forget over a few to a thousand tokens
    s["g"] = -torch.exp(-1 - 6 * uni(Hv)) * (0.2 + 2 * uni(B, S, Hv))
    s["beta"] = torch.sigmoid(rn(B, S, Hv))
    s["state"] = 0.3 * rn(B, Hv, Dk, Dv)
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(0, S + 1, (B,), device=dev, generator=g, dtype=torch.int32)
        s["lengths"][0] = S
    if op == "delta":
        s["o"] = torch.zeros(B, S, Hv, Dv, dtype=dt, device=dev)  # rows behind a sequence's end stay as they are
        s["last"] = torch.empty(B, Hv, Dk, Dv, device=dev)
    else:
        s["do"] = (0.1 * rn(B, S, Hv, Dv)).to(dt)
        s["dlast"] = 0.1 * rn(B, Hv, Dk, Dv)
    return s


# -------------------------------------------------------------- plain forms


def _plain_quant(y, group):
    """(q, scale): q = round(y / scale) with scale = the group's largest magnitude / 448."""
    T, C = y.shape
    width = group or C
    n = -(-C // width)
    if n * width != C:
        y = torch.cat([y, torch.zeros(T, n * width - C, device=y.device)], 1)
    v = y.view(T, n, width)
    scale = v.abs().amax(2) / F8_MAX
    scale = torch.where(scale < TINY, 1.0, scale)
    q = (v / scale[:, :, None]).clamp(-F8_MAX, F8_MAX).view(T, n * width)[:, :C]
    return q.to(torch.float8_e4m3fn), scale


def _plain_norm(v, s, case, dt):
    d = v - v.mean(1, keepdim=True)
    y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS) * s["weight"] + s["bias"]
    if case["quant"]:
        return (v.to(dt),) + _plain_quant(y, case["group"])
    return v.to(dt), y.to(dt)


def _plain_norm_backward(s):
    v, dy = s["s"].float(), s["dy"].float()
    d = v - v.mean(1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    n = d * rstd
    wdy = s["weight"] * dy
    dx = rstd * (wdy - wdy.mean(1, keepdim=True) - n * (wdy * n).mean(1, keepdim=True)) + s["ds"].float()
    return dx.to(s["s"].dtype), (dy * n).sum(0), dy.sum(0)


def _chunks(s, case):
    """The inputs in float32 as [B, Hv, chunks, CHUNK, ...], tokens behind a length and the last chunk's
    end neutral, with what every chunk can do by itself: the decays and the inverse of its triangle."""
    B, S, Hk, Hv = (case[v] for v in ("B", "S", "Hk", "Hv"))
    n = -(-S // CHUNK)
    live = torch.ones(B, S, device="cuda", dtype=torch.bool)
    if s["lengths"] is not None:
        live = torch.arange(S, device="cuda")[None] < s["lengths"][:, None]

    def cut(t):
        t = torch.where(live.view(B, S, *[1] * (t.dim() - 2)), t.float(), 0.0)
        t = torch.cat([t, t.new_zeros(B, n * CHUNK - S, *t.shape[2:])], 1)
        if t.shape[2] != Hv:
            t = t.repeat_interleave(Hv // Hk, 2)
        return t.transpose(1, 2).reshape(B, Hv, n, CHUNK, *t.shape[3:])

    q, k, v, g, beta = (cut(s[x]) for x in ("q", "k", "v", "g", "beta"))
    G = g.double().cumsum(3)
    low = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    D = torch.where(low, (G[..., :, None] - G[..., None, :]).float(), -math.inf).exp()
    KK = (k @ k.transpose(3, 4)) * D * torch.ones_like(low).tril(-1)
    A = KK * beta[..., None, :]
    inv = torch.eye(CHUNK, device="cuda").expand_as(A).contiguous()
    for i in range(1, CHUNK):
        inv[..., i:i + 1, :i] = -(A[..., i:i + 1, :i] @ inv[..., :i, :i])
    P = (q @ k.transpose(3, 4)) * D
    ahead, to_end = G.float().exp(), (G[..., -1:] - G).float().exp()
    return dict(q=q, k=k, v=v, beta=beta, D=D, KK=KK, inv=inv, P=P, ahead=ahead, to_end=to_end, live=live, n=n, cut=cut)


def _walk(c, state, keep):
    """Outputs (without the scale) and the last state; with `keep` every chunk's first state and z."""
    S0, outs, kept = state, [], []
    for i in range(c["n"]):
        q, k, ahead = c["q"][:, :, i], c["k"][:, :, i], c["ahead"][:, :, i, :, None]
        z = c["inv"][:, :, i] @ (c["v"][:, :, i] - ahead * (k @ S0))
        x = c["beta"][:, :, i, :, None] * z
        if keep:
            kept.append((S0, z))
        else:
            outs.append(ahead * (q @ S0) + c["P"][:, :, i] @ x)
        S0 = ahead[:, :, -1:] * S0 + k.transpose(2, 3) @ (c["to_end"][:, :, i, :, None] * x)
    return kept if keep else (torch.stack(outs, 2), S0)


def _uncut(t, case):
    B, S, Hv = case["B"], case["S"], case["Hv"]
    return t.reshape(B, Hv, -1, *t.shape[4:])[:, :, :S].transpose(1, 2)


def _plain_steps(s, case):
    """Token by token, for a few tokens: the chunks' triangles would cost more than the recurrence."""
    B, S, per, scale = case["B"], case["S"], case["Hv"] // case["Hk"], case["Dk"] ** -0.5
    q, k = (s[x].float().repeat_interleave(per, 2)[..., None] for x in ("q", "k"))
    v, alpha, M = s["v"].float(), s["g"].exp()[..., None, None], s["state"]
    beta = s["beta"][..., None]
    o = torch.zeros_like(v)
    for t in range(S):
        F = alpha[:, t] * M
        new = F + k[:, t] * (beta[:, t] * (v[:, t] - (F * k[:, t]).sum(2)))[:, :, None]
        out = (new * q[:, t]).sum(2) * scale
        if s["lengths"] is not None:
            on = (t < s["lengths"])[:, None, None]
            new, out = torch.where(on[..., None], new, M), torch.where(on, out, 0.0)
        M, o[:, t] = new, out
    return o.to(s["v"].dtype), M


def _plain_delta(s, case):
    if case["S"] <= 16:
        return _plain_steps(s, case)
    c = _chunks(s, case)
    o, last = _walk(c, s["state"], False)
    o = torch.where(c["live"][:, :, None, None], _uncut(o * case["Dk"] ** -0.5, case), 0.0)
    return o.to(s["v"].dtype), last


def _plain_delta_backward(s, case):
    scale = case["Dk"] ** -0.5
    c = _chunks(s, case)
    do = c["cut"](s["do"]) * scale
    kept = _walk(c, s["state"], True)
    dS = s["dlast"]
    low = torch.ones(CHUNK, CHUNK, device="cuda").tril()
    dq, dk, dv, dG, db = ([None] * c["n"] for _ in range(5))
    for i in reversed(range(c["n"])):
        q, k, beta, D, P, KK = (c[x][:, :, i] for x in ("q", "k", "beta", "D", "P", "KK"))
        ahead, to_end, d = c["ahead"][:, :, i, :, None], c["to_end"][:, :, i, :, None], do[:, :, i]
        S0, z = kept[i]
        dx = P.transpose(2, 3) @ d + to_end * (k @ dS)
        w = c["inv"][:, :, i].transpose(2, 3) @ (beta[..., None] * dx)
        x = beta[..., None] * z
        dP = (d @ x.transpose(2, 3)) * D
        dA = -(w @ x.transpose(2, 3)) * D * low.tril(-1)
        dq1 = ahead * (d @ S0.transpose(2, 3)) + dP @ k
        late = -ahead * (w @ S0.transpose(2, 3)) + dA @ k  # k of a token as it reads
        early = to_end * (x @ dS.transpose(2, 3))  # k of a token as it is written
        into = early + dP.transpose(2, 3) @ q + dA.transpose(2, 3) @ k
        dq[i], dk[i], dv[i] = dq1, late + into, w
        db[i] = (z * dx).sum(3) - (KK * (w @ z.transpose(2, 3))).sum(2)
        dGi = (q * dq1 + k * late - k * into).sum(3)
        dGi[..., -1] += (k * early).sum((2, 3)) + (ahead[:, :, -1:] * S0 * dS).sum((2, 3))
        dG[i] = dGi
        dS = ahead[:, :, -1:] * dS + (ahead * q).transpose(2, 3) @ d - (ahead * k).transpose(2, 3) @ w
    dg = torch.stack(dG, 2).flip(3).cumsum(3).flip(3)
    B, S, Hk, Hv = (case[v] for v in ("B", "S", "Hk", "Hv"))
    dt = s["v"].dtype
    out = []
    for t, shared in ((dq, True), (dk, True), (dv, False), (dg, False), (db, False)):
        t = _uncut(t if torch.is_tensor(t) else torch.stack(t, 2), case)
        t = torch.where(c["live"].view(B, S, *[1] * (t.dim() - 2)), t, 0.0)
        out.append(t.reshape(B, S, Hk, Hv // Hk, -1).sum(3) if shared else t)
    return out[0].to(dt), out[1].to(dt), out[2].to(dt), out[3], out[4], dS


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "norm":
        return _plain_norm(s["x"].float() + s["residual"].float(), s, case, s["x"].dtype)
    if op == "pre_norm":
        return _plain_norm((s["h_pre"][:, :, None] * s["X"].float()).sum(1), s, case, s["X"].dtype)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    if op == "delta":
        return _plain_delta(s, case)
    return _plain_delta_backward(s, case)


def _own(s, case, op):
    import stream_residual_mixing_amd as hc

    quant = torch.float8_e4m3fn if case.get("quant") else None
    if op == "norm":
        r = hc.hc_layer_norm(s["x"], s["weight"], s["bias"], EPS, residual=s["residual"], quant=quant,
                             group=case["group"])
        return (r["s"], r["y"]) + ((r["scale"],) if quant else ())
    if op == "pre_norm":
        r = hc.hc_pre_layer_norm(s["X"], s["h_pre"], s["weight"], s["bias"], EPS, quant=quant, group=case["group"])
        return (r["F_in"], r["y"]) + ((r["scale"],) if quant else ())
    if op == "norm_backward":
        return hc.hc_layer_norm_backward(s["s"], s["weight"], s["dy"], EPS, ds=s["ds"])
    if op == "delta":
        return hc.hc_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], lengths=s["lengths"],
                                 out=(s["o"], s["last"]))
    return hc.hc_gated_delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["state"], s["dlast"],
                                      lengths=s["lengths"])


# --------------------------------------------------------------------- work


def work(case):
    """Each input read once and each output written once; the recurrence's products token by token."""
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("norm", "pre_norm"):
        T, C = case["T"], case["C"]
        reads = 2 if op == "norm" else case["n"]
        outs = e + (1 if case["quant"] else e)
        scales = 4 * T * -(-C // (case["group"] or C)) if case["quant"] else 0
        return {"bytes": T * C * (reads * e + outs) + scales + 8 * C, "flops": T * C * (2 * reads + 8)}
    if op == "norm_backward":
        T, C = case["T"], case["C"]
        return {"bytes": T * C * 4 * e + 12 * C, "flops": T * C * 18}
    B, S, Hk, Hv, Dk, Dv = (case[v] for v in ("B", "S", "Hk", "Hv", "Dk", "Dv"))
    n, state = B * S, 4 * B * Hv * Dk * Dv
    if op == "delta":
        return {"bytes": n * (2 * Hk * Dk + 2 * Hv * Dv) * e + 8 * n * Hv + 2 * state, "flops": n * Hv * Dk * Dv * 7}
    return {"bytes": n * (4 * Hk * Dk + 3 * Hv * Dv) * e + 16 * n * Hv + 3 * state, "flops": n * Hv * Dk * Dv * 21}


# -------------------------------------------------- the definition in float64


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("norm", "pre_norm"):
        if op == "norm":
            v = s["x"].to(f64) + s["residual"].to(f64)
        else:
            v = torch.zeros(case["T"], case["C"], dtype=f64, device="cuda")
            for i in range(case["n"]):
                v += s["h_pre"][:, i:i + 1].to(f64) * s["X"][:, i].to(f64)
        mean = v.sum(1, keepdim=True) / case["C"]
        var = ((v - mean) ** 2).sum(1, keepdim=True) / case["C"]
        y = (v - mean) / (var + EPS) ** 0.5 * s["weight"].to(f64) + s["bias"].to(f64)
        if not case["quant"]:
            return v, y
        width = case["group"] or case["C"]
        parts = [y[:, c:c + width] for c in range(0, case["C"], width)]
        scales = [p.abs().max(1, keepdim=True).values / F8_MAX for p in parts]
        return v, torch.cat([p / sc for p, sc in zip(parts, scales)], 1), torch.cat(scales, 1)
    if op == "norm_backward":
        v, dy, w = s["s"].to(f64), s["dy"].to(f64), s["weight"].to(f64)
        C = case["C"]
        c = v - v.sum(1, keepdim=True) / C
        sd = ((c ** 2).sum(1, keepdim=True) / C + EPS) ** 0.5
        up = w * dy
        dx = (up - up.sum(1, keepdim=True) / C) / sd - c * (c * up).sum(1, keepdim=True) / (C * sd ** 3)
        return dx + s["ds"].to(f64), (dy * c / sd).sum(0), dy.sum(0)
    B, S, Hk, Hv, Dk, Dv = (case[v] for v in ("B", "S", "Hk", "Hv", "Dk", "Dv"))
    per = Hv // Hk
    scale = Dk ** -0.5
    head = lambda t: t.to(f64).repeat_interleave(per, 2)  # noqa: E731
    q, k, v = head(s["q"]), head(s["k"]), s["v"].to(f64)
    alpha, beta = torch.exp(s["g"].to(f64)), s["beta"].to(f64)
    on = torch.ones(B, S, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        on = torch.arange(S, device="cuda")[None] < s["lengths"][:, None].to(torch.int64)

    def step(M, t):
        """The state after token t, the decayed one before it, and the token's surprise."""
        m = on[:, t, None, None, None]
        F = alpha[:, t, :, None, None] * M
        z = v[:, t] - (F * k[:, t, :, :, None]).sum(2)
        new = F + k[:, t, :, :, None] * (beta[:, t, :, None] * z)[:, :, None]
        return torch.where(m, new, M), F, z

    M = s["state"].to(f64)
    if op == "delta":
        o = torch.zeros(B, S, Hv, Dv, dtype=f64, device="cuda")
        for t in range(S):
            M, _, _ = step(M, t)
            o[:, t] = torch.where(on[:, t, None, None], scale * (M * q[:, t, :, :, None]).sum(2), 0.0)
        return o, M
    marks, every = [], max(1, int(S ** 0.5))
    for t in range(S):  # the states of every few tokens; those between are formed again on the way back
        if t % every == 0:
            marks.append(M)
        M, _, _ = step(M, t)
    do = s["do"].to(f64)
    R = s["dlast"].to(f64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(alpha), torch.zeros_like(beta)
    for b in reversed(range(len(marks))):
        M, seg = marks[b], []
        for t in range(b * every, min(S, (b + 1) * every)):
            M, F, z = step(M, t)
            seg.append((t, M, F, z))
        for t, after, F, z in reversed(seg):
            m = on[:, t]
            kt, d = k[:, t, :, :, None], scale * do[:, t, :, None]
            dM = R + q[:, t, :, :, None] * d
            into = (dM * kt).sum(2)
            dz = beta[:, t, :, None] * into
            dF = dM - kt * dz[:, :, None]
            dq[:, t] = torch.where(m[:, None, None], (after * d).sum(3), 0.0)
            dk[:, t] = torch.where(m[:, None, None],
                                   (dM * (beta[:, t, :, None] * z)[:, :, None] - F * dz[:, :, None]).sum(3), 0.0)
            dv[:, t] = torch.where(m[:, None, None], dz, 0.0)
            db[:, t] = torch.where(m[:, None], (into * z).sum(2), 0.0)
            dg[:, t] = torch.where(m[:, None], (dF * F).sum((2, 3)), 0.0)
            R = torch.where(m[:, None, None, None], alpha[:, t, :, None, None] * dF, R)
    fold = lambda t: t.view(B, S, Hk, per, Dk).sum(3)  # noqa: E731
    return fold(dq), fold(dk), dv, dg, db, R
