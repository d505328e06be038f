"""The sublayer operators beside the stream mixing, as measurable cases.

Four operators of hc.h, each with its gradient: the root-mean-square norm in
front of a sublayer function (with the residual's addition or the pre-read of the
streams, and an 8-bit output), the gated linear recurrence over the sequence
inside it, the balance loss of the stream router, and the router's own backward.

run() computes a case's operator once: in plain float32 torch operations, or with
`own` set through the package. exact() is the definition in float64.
"""
import math

import torch

own = False

F8_MAX = 448.0  # largest finite e4m3
TINY = 2.0 ** -126  # smallest normal float32: a smaller scale is replaced by 1
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # serving, one decode step of 16 requests: the residual joins and the projections read 8 bits, one
        # scale a token; latency counts
        dict(name="norm_decode", op="norm", T=16, C=4096, dtype="bf16", quant="e4m3", group=0),
        # a prefill chunk: the same call with a scale for each 128 channels
        dict(name="norm_prefill", op="norm", T=8192, C=4096, dtype="bf16", quant="e4m3", group=128),
        # training forward at the widest state: pre-read of 4 streams and norm in one pass, F_in kept for the backward
        dict(name="pre_norm_wide", op="pre_norm", T=16384, n=4, C=7168, dtype="bf16", quant="", group=0),
        # its backward at the common width, with the residual's own gradient joined, an odd number of tokens
        dict(name="norm_backward", op="norm_backward", T=8191, C=4096, dtype="bf16"),
        # serving, one new token for each of 64 sequences
        dict(name="scan_step", op="scan", B=64, S=1, C=4096, dtype="bf16", tied=True, ragged=False),
        # one long sequence, training forward
        dict(name="scan_long", op="scan", B=1, S=8192, C=4096, dtype="bf16", tied=True, ragged=False),
        # a padded batch in float32, odd sizes, the untied form
        dict(name="scan_padded", op="scan", B=5, S=1021, C=1100, dtype="f32", tied=False, ragged=True),
        # training backward of two sequences
        dict(name="scan_backward", op="scan_backward", B=2, S=4096, C=4096, dtype="bf16", tied=True, ragged=False),
        # router loss and its gradient: a fine-tuning microbatch and the common batch
        dict(name="balance_small", op="balance", B=1, S=509, N=8, k=4, m=1, padded=False),
        dict(name="balance_batch", op="balance", B=8, S=4096, N=16, k=4, m=2, padded=True),
        # router weights' and state's gradients: a small width with an odd token count, the common width
        dict(name="router_backward_small", op="router_backward", T=1021, N=8, m=2, C=512),
        dict(name="router_backward", op="router_backward", T=8192, N=16, m=2, C=4096),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pre_norm", "norm_backward", "scan", "scan", "scan_backward", "balance",
                     "router_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "pre_norm"):
        quant = rng.choice(["", "e4m3"])
        c = dict(op=op, T=_log(rng, 1, 16384), C=_log(rng, 64, 8192), dtype=dtype, quant=quant,
                 group=rng.choice([0, 32, 64, 128]) if quant else 0)
        if rng.random() < 0.6:
            c["C"] = max(128, c["C"] // 128 * 128)
        if op == "pre_norm":
            c.update(n=rng.choice([2, 4, 4, 8]), T=_log(rng, 1, 8192))
        return c
    if op == "norm_backward":
        C = _log(rng, 64, 8192)
        return dict(op=op, T=_log(rng, 1, 16384), C=max(128, C // 128 * 128) if rng.random() < 0.6 else C, dtype=dtype)
    if op in ("scan", "scan_backward"):
        B, C = _log(rng, 1, 64), _log(rng, 64, 8192)
        S = _log(rng, 1, max(1, min(16384, (1 << 25) // (B * C))))
        return dict(op=op, B=B, S=S, C=max(64, C // 64 * 64) if rng.random() < 0.6 else C, dtype=dtype,
                    tied=rng.random() < 0.5, ragged=rng.random() < 0.3)
    if op == "balance":
        N = rng.choice([4, 8, 12, 16])
        k = rng.randint(2, min(N - 1, 6))
        B = _log(rng, 1, 16)
        return dict(op=op, B=B, S=_log(rng, 1, 65536 // B), N=N, k=k, m=rng.randint(1, k - 1),
                    padded=rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 1, 4096), N=rng.choice([4, 8, 12, 16]), m=rng.randint(1, 3),
                C=32 * _log(rng, 2, 128))


# ------------------------------------------------------------------ inputs


def _quant_dtype(case):
    return torch.float8_e4m3fn if case["quant"] else None


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    rn = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    uni = lambda *s: torch.rand(*s, device=dev, generator=g)  # noqa: E731
    op, s = case["op"], {"case": case}
    if op == "norm":
        dt = DT[case["dtype"]]
        # a residual stream grows over the layers, some channels far beyond the others
        s["residual"] = (4 * rn(case["T"], case["C"]) * torch.exp(0.7 * rn(case["C"]))).to(dt)
        s["x"] = rn(case["T"], case["C"]).to(dt)
        s["weight"] = 1 + 0.2 * rn(case["C"])
    elif op == "pre_norm":
        dt = DT[case["dtype"]]
        s["X"] = torch.empty(case["T"], case["n"], case["C"], dtype=dt, device=dev).normal_(generator=g)
        s["h_pre"] = torch.sigmoid(rn(case["T"], case["n"]))
        s["weight"] = 1 + 0.2 * rn(case["C"])
    elif op == "norm_backward":
        dt = DT[case["dtype"]]
        s["s"] = (2 * rn(case["T"], case["C"])).to(dt)
        s["dy"] = (0.1 * rn(case["T"], case["C"])).to(dt)
        s["ds"] = (0.1 * rn(case["T"], case["C"])).to(dt)
        s["weight"] = 1 + 0.2 * rn(case["C"])
    elif op in ("scan", "scan_backward"):
        dt, B, S, C = DT[case["dtype"]], case["B"], case["S"], case["C"]
        s["x"] = rn(B, S, C).to(dt)
        # channels forget over a few to a thousand tokens
        s["gate"] = (6 * uni(C) + 1 + rn(B, S, C)).to(dt)
        s["h0"] = rn(B, C)
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(0, S + 1, (B,), device=dev, generator=g, dtype=torch.int32)
            s["lengths"][0] = S
        if op == "scan":
            s["y"] = torch.zeros(B, S, C, dtype=dt, device=dev)  # rows behind a sequence's end stay as they are
            s["h_last"] = torch.empty(B, C, device=dev)
        else:
            y, _ = _plain_scan(s["x"], s["gate"], s["h0"], s["lengths"], case["tied"])
            s["y"] = y
            s["dy"] = (0.1 * rn(B, S, C)).to(dt)
            s["dh_last"] = 0.1 * rn(B, C)
    elif op == "balance":
        B, S, N, k, m = (case[v] for v in ("B", "S", "N", "k", "m"))
        T, E = B * S, N - m
        s["score"] = torch.sigmoid(0.8 * rn(T, E) + 0.5 * rn(E))
        top = torch.topk(s["score"], k - m, dim=1).indices + m
        fixed = torch.arange(m, device=dev).expand(T, m)
        s["idx"] = torch.sort(torch.cat([fixed, top], 1), 1).values.to(torch.int32).contiguous()
        s["mask"] = None
        if case["padded"]:
            n = torch.randint(0, S + 1, (B, 1), device=dev, generator=g)
            s["mask"] = (torch.arange(S, device=dev)[None] < n).reshape(T).contiguous()
        s["dloss"] = 0.5 + uni(1)
    else:
        T, N, m, C = (case[v] for v in ("T", "N", "m", "C"))
        E = N - m
        s["X"] = torch.empty(T, N, C, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        s["dX"] = torch.empty(T, N, C, dtype=torch.bfloat16, device=dev).normal_(0, 0.02, generator=g)
        s["w_router"] = rn(N * C, E) * (2.0 / math.sqrt(N * C))  # logits of size 2
        x = s["X"].view(T, N * C).float()
        s["score"] = torch.sigmoid((x @ s["w_router"]) / x.square().mean(1, keepdim=True).sqrt())
        s["dscore"] = 0.02 * rn(T, E)
        s["out"] = torch.empty_like(s["dX"])
    return s


# -------------------------------------------------------------- plain forms


def _plain_quant(y, quant, group):
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


def _plain_norm(v, weight, eps, case, dt):
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + eps) * weight
    if case["quant"]:
        return _plain_quant(y, case["quant"], case["group"])
    return (y.to(dt),)


def _plain_scan(x, gate, h0, lengths, tied):
    """y and the last state, by doubling: after step d every token holds the map over its last 2d tokens.
    The loop has log2(S) steps, each over the whole array."""
    B, S, C = x.shape
    a = torch.sigmoid(gate.float())
    b = (torch.sigmoid(-gate.float()) if tied else 1.0) * x.float()
    if lengths is not None:
        live = torch.arange(S, device=x.device)[None, :, None] < lengths[:, None, None]
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    b[:, 0] += a[:, 0] * h0
    d = 1
    while d < S:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    last = b[:, -1].clone()
    if lengths is not None:
        b = torch.where(live, b, 0.0)
    return b.to(x.dtype), last


def _plain_scan_backward(x, gate, y, dy, h0, dh_last, lengths, tied):
    B, S, C = x.shape
    x32, y32 = x.float(), y.float()
    a, u = torch.sigmoid(gate.float()), torch.sigmoid(-gate.float())
    g = dy.float()
    step = a
    if lengths is not None:
        live = torch.arange(S, device=x.device)[None, :, None] < lengths[:, None, None]
        step, g = torch.where(live, a, 1.0), torch.where(live, g, 0.0)
    # the last state's gradient enters at the last token; tokens behind a sequence's end pass it on (step 1)
    carry = torch.cat([step[:, 1:], torch.ones_like(step[:, :1])], 1)
    g[:, -1] += dh_last
    d = 1
    while d < S:
        g = torch.cat([g[:, :-d] + carry[:, :-d] * g[:, d:], g[:, -d:]], 1)
        carry = torch.cat([carry[:, :-d] * carry[:, d:], carry[:, -d:]], 1)
        d *= 2
    dh0 = step[:, 0] * g[:, 0]
    prev = torch.cat([h0[:, None], y32[:, :-1]], 1)
    dx = (u if tied else 1.0) * g
    dgate = g * (prev - x32 if tied else prev) * (a * u)
    if lengths is not None:
        dx, dgate = torch.where(live, dx, 0.0), torch.where(live, dgate, 0.0)
    return dx.to(x.dtype), dgate.to(x.dtype), dh0


def _plain_balance(s, case):
    B, S, N, k, m = (case[v] for v in ("B", "S", "N", "k", "m"))
    E = N - m
    live = torch.ones(B, S, device="cuda", dtype=torch.bool) if s["mask"] is None else s["mask"].view(B, S)
    score = torch.where(live[:, :, None], s["score"].view(B, S, E), 0.0)
    total = score.sum(2, keepdim=True)
    p = torch.where(total > 0, score / total, 0.0)
    tokens = live.sum(1)
    hit = (s["idx"].view(B, S, k, 1) == torch.arange(N, device="cuda")) & live[:, :, None, None]
    count = hit.sum((1, 2))
    n = tokens.clamp(min=1).float()[:, None]
    mean_p = p.sum(1) / n
    f = count[:, m:].float() * (E / (k - m)) / n
    loss = (f * mean_p).sum() / B
    scale = s["dloss"] / (B * n[:, :, None])
    grad = scale * (f[:, None] - (f[:, None] * p).sum(2, keepdim=True)) / total
    dscore = torch.where(live[:, :, None] & (total > 0), grad, 0.0).view(B * S, E)
    return loss, count.to(torch.int32), tokens.to(torch.int32), mean_p, dscore


def _plain_router_backward(s, case):
    T, N, C = s["X"].shape
    x = s["X"].float().view(T, N * C)
    r = x.square().mean(1, keepdim=True).sqrt()
    sc = s["score"]
    dz = s["dscore"] * sc * (1 - sc)
    z = torch.log(sc) - torch.log1p(-sc)
    along = (dz * torch.where(dz != 0, z, 0.0)).sum(1, keepdim=True) / (N * C)
    dxr = (dz / r) @ s["w_router"].t() - (along / r.square()) * x
    dw = x.t() @ (dz / r)
    return (s["dX"].float().view(T, N * C) + dxr).to(torch.bfloat16).view(T, N, C), dw


EPS = 1e-6


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "norm":
        v = s["x"].float() + s["residual"].float()
        return (v.to(s["x"].dtype),) + _plain_norm(v, s["weight"], EPS, case, s["x"].dtype)
    if op == "pre_norm":
        v = (s["h_pre"][:, :, None] * s["X"].float()).sum(1)
        return (v.to(s["X"].dtype),) + _plain_norm(v, s["weight"], EPS, case, s["X"].dtype)
    if op == "norm_backward":
        v, dy = s["s"].float(), s["dy"].float()
        rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
        vh = v * rstd
        wdy = s["weight"] * dy
        dx = rstd * (wdy - vh * (wdy * vh).mean(1, keepdim=True)) + s["ds"].float()
        return dx.to(s["s"].dtype), (dy * vh).sum(0)
    if op == "scan":
        return _plain_scan(s["x"], s["gate"], s["h0"], s["lengths"], case["tied"])
    if op == "scan_backward":
        return _plain_scan_backward(s["x"], s["gate"], s["y"], s["dy"], s["h0"], s["dh_last"], s["lengths"],
                                    case["tied"])
    if op == "balance":
        return _plain_balance(s, case)
    return _plain_router_backward(s, case)


def _own(s, case, op):
    import stream_residual_mixing_amd as hc

    if op == "norm":
        r = hc.hc_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], quant=_quant_dtype(case),
                           group=case["group"])
        return (r["s"], r["y"]) + ((r["scale"],) if case["quant"] else ())
    if op == "pre_norm":
        r = hc.hc_pre_norm(s["X"], s["h_pre"], s["weight"], EPS, quant=_quant_dtype(case), group=case["group"])
        return (r["F_in"], r["y"]) + ((r["scale"],) if case["quant"] else ())
    if op == "norm_backward":
        return hc.hc_rms_norm_backward(s["s"], s["weight"], s["dy"], EPS, ds=s["ds"])
    if op == "scan":
        return hc.hc_gated_scan(s["x"], s["gate"], s["h0"], lengths=s["lengths"], tied=case["tied"],
                                out=(s["y"], s["h_last"]))
    if op == "scan_backward":
        return hc.hc_gated_scan_backward(s["x"], s["gate"], s["y"], s["dy"], s["h0"], s["dh_last"],
                                         lengths=s["lengths"], tied=case["tied"])
    if op == "balance":
        r = hc.xhc_balance_loss(s["score"], s["idx"], case["B"], case["S"], m=case["m"], mask=s["mask"])
        dscore = hc.xhc_balance_loss_backward(s["score"], r["count"], r["tokens"], case["k"], case["B"], case["S"],
                                              dloss=s["dloss"], mask=s["mask"])
        return r["loss"], r["count"], r["tokens"], r["mean_p"], dscore
    return hc.xhc_router_backward(s["X"], s["w_router"], s["score"], s["dscore"], s["dX"], out=s["out"])


# --------------------------------------------------------------------- work


def work(case):
    """Each input read once and each output written once."""
    op = case["op"]
    if op in ("norm", "pre_norm"):
        T, C, e = case["T"], case["C"], SIZE[case["dtype"]]
        reads = 2 if op == "norm" else case["n"]
        outs = e + (1 if case["quant"] else e)
        scales = 4 * T * -(-C // (case["group"] or C)) if case["quant"] else 0
        return {"bytes": T * C * (reads * e + outs) + scales + 4 * C, "flops": T * C * (2 * reads + 6)}
    if op == "norm_backward":
        T, C, e = case["T"], case["C"], SIZE[case["dtype"]]
        return {"bytes": T * C * 4 * e + 8 * C, "flops": T * C * 14}
    if op == "scan":
        n, e = case["B"] * case["S"] * case["C"], SIZE[case["dtype"]]
        return {"bytes": n * 3 * e + 8 * case["B"] * case["C"], "flops": n * 12}
    if op == "scan_backward":
        n, e = case["B"] * case["S"] * case["C"], SIZE[case["dtype"]]
        return {"bytes": n * 6 * e + 12 * case["B"] * case["C"], "flops": n * 16}
    if op == "balance":
        T, E = case["B"] * case["S"], case["N"] - case["m"]
        return {"bytes": T * (8 * E + 4 * case["k"] + (1 if case["padded"] else 0)), "flops": T * E * 10}
    n, E = case["T"] * case["N"] * case["C"], case["N"] - case["m"]
    return {"bytes": n * 6 + 8 * case["N"] * case["C"] * E + 8 * case["T"] * E, "flops": n * (4 * E + 6)}


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
        norm = (v ** 2).sum(1, keepdim=True) / case["C"] + EPS
        y = v / norm ** 0.5 * s["weight"].to(f64)
        if not case["quant"]:
            return v, y
        width = case["group"] or case["C"]
        parts = [y[:, c:c + width] for c in range(0, case["C"], width)]
        scales = [p.abs().max(1, keepdim=True).values / F8_MAX for p in parts]
        return v, torch.cat([p / sc for p, sc in zip(parts, scales)], 1), torch.cat(scales, 1)
    if op == "norm_backward":
        v, dy, w = s["s"].to(f64), s["dy"].to(f64), s["weight"].to(f64)
        n2 = (v ** 2).sum(1, keepdim=True) / case["C"] + EPS
        inner = (v * dy * w).sum(1, keepdim=True) / case["C"]
        return (w * dy / n2 ** 0.5 - v * inner / n2 ** 1.5 + s["ds"].to(f64),
                (dy * v / n2 ** 0.5).sum(0))
    if op == "scan":
        a = 1 / (1 + torch.exp(-s["gate"].to(f64)))
        u = (1 - a if case["tied"] else torch.ones_like(a)) * s["x"].to(f64)
        h, y = s["h0"].to(f64), torch.zeros_like(a)
        ends = torch.full((case["B"],), case["S"], device="cuda") if s["lengths"] is None else s["lengths"]
        for t in range(case["S"]):
            new = a[:, t] * h + u[:, t]
            if s["lengths"] is None:
                h = y[:, t] = new
            else:
                on = (t < ends)[:, None]
                h = torch.where(on, new, h)
                y[:, t] = torch.where(on, new, 0.0)
        return y, h
    if op == "scan_backward":
        a = 1 / (1 + torch.exp(-s["gate"].to(f64)))
        x, y, dy = s["x"].to(f64), s["y"].to(f64), s["dy"].to(f64)
        g = s["dh_last"].to(f64)
        dx, dgate = torch.zeros_like(x), torch.zeros_like(x)
        for t in range(case["S"] - 1, -1, -1):
            on = torch.ones(case["B"], 1, dtype=torch.bool, device="cuda") if s["lengths"] is None else (
                t < s["lengths"])[:, None]
            dh = dy[:, t] + g
            h = y[:, t - 1] if t else s["h0"].to(f64)
            da = dh * (h - x[:, t]) if case["tied"] else dh * h
            dx[:, t] = torch.where(on, dh * (1 - a[:, t]) if case["tied"] else dh, 0.0)
            dgate[:, t] = torch.where(on, da * a[:, t] * (1 - a[:, t]), 0.0)
            g = torch.where(on, dh * a[:, t], g)
        return dx, dgate, g
    if op == "balance":
        B, S, N, k, m = (case[v] for v in ("B", "S", "N", "k", "m"))
        E = N - m
        score = s["score"].to(f64).view(B, S, E)
        loss, dscore = torch.zeros((), dtype=f64, device="cuda"), torch.zeros_like(score)
        counts, ntok, means = [], [], []
        for b in range(B):
            on = torch.ones(S, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].view(B, S)[b]
            p = score[b][on] / score[b][on].sum(1, keepdim=True)
            c = torch.bincount(s["idx"].view(B, S, k)[b][on].reshape(-1).long(), minlength=N)
            n = max(1, int(on.sum()))
            f = c[m:].to(f64) * E / ((k - m) * n)
            loss += (f * p.sum(0) / n).sum() / B
            dscore[b][on] = float(s["dloss"]) / (B * n) * (f - (p * f).sum(1, keepdim=True)) / score[b][on].sum(
                1, keepdim=True)
            counts.append(c.to(torch.int32))
            ntok.append(int(on.sum()))
            means.append(p.sum(0) / n)
        return (loss, torch.stack(counts), torch.tensor(ntok, dtype=torch.int32), torch.stack(means),
                dscore.view(B * S, E))
    T, N, m, C = (case[v] for v in ("T", "N", "m", "C"))
    w = s["w_router"].to(f64)
    outs, dw = [], torch.zeros_like(w)
    for i in range(0, T, 512):  # 512 tokens' float64 copies at a time
        x = s["X"][i:i + 512].to(f64).view(-1, N * C)
        sc = s["score"][i:i + 512].to(f64)
        dz = s["dscore"][i:i + 512].to(f64) * sc * (1 - sc)
        n2 = (x ** 2).sum(1, keepdim=True) / (N * C)
        z = torch.where(dz != 0, torch.log(sc / (1 - sc)), 0.0)  # a score of 0 or 1 passes nothing on
        along = (dz * z).sum(1, keepdim=True)
        dx = dz @ w.t() / n2 ** 0.5 - x * along / (n2 * N * C)
        outs.append((s["dX"][i:i + 512].to(f64).view(-1, N * C) + dx).view(-1, N, C))
        dw += x.t() @ (dz / n2 ** 0.5)
    return torch.cat(outs), dw
