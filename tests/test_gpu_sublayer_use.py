"""The norm, scan and router calls as a program uses them: captured and replayed, on
other streams, several at once, with the same results every time, on arrays past 2^31
elements, and together with the stream mixing in a forward and backward step."""
import numpy as np
import pytest

from hc_testutil import have_gpu, note

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc


def _inputs(seed, B=2, S=700, C=512, N=8, k=4, m=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    T, E = B * S, N - m
    score = torch.sigmoid(rn(T, E))
    idx = torch.cat([torch.arange(m, device="cuda").expand(T, m), m + torch.topk(score, k - m, 1).indices], 1)
    return dict(x=rn(T, C).bfloat16(), r=rn(T, C).bfloat16(), w=1 + 0.1 * rn(C), gate=(3 + rn(B, S, C)).bfloat16(),
                h0=rn(B, C), dy=rn(B, S, C).bfloat16(), dl=rn(B, C), X=rn(T, N, C).bfloat16(), score=score,
                idx=idx.sort(1).values.int().contiguous(), wr=0.05 * rn(N * C, E), dX=rn(T, N, C).bfloat16(),
                L=torch.tensor([S, S // 3], dtype=torch.int32, device="cuda"), h=torch.sigmoid(rn(T, N)), B=B, S=S,
                k=k, m=m)


def _step(i, stream=None):
    """Every new call once; all outputs."""
    B, S, k, m = i["B"], i["S"], i["k"], i["m"]
    C = i["x"].shape[1]
    o = {"stream": stream}
    a = hc.hc_rms_norm(i["x"], i["w"], residual=i["r"], **o)
    q = hc.hc_rms_norm(i["x"], i["w"], residual=i["r"], quant=torch.float8_e4m3fn, group=128, **o)
    p = hc.hc_pre_norm(i["X"], i["h"], i["w"], **o)
    y0 = torch.zeros(B, S, C, dtype=torch.bfloat16, device="cuda")
    x = a["y"].view(B, S, C)
    y, last = hc.hc_gated_scan(x, i["gate"], i["h0"], lengths=i["L"], out=(y0, None), **o)
    dx, dg, dh0 = hc.hc_gated_scan_backward(x, i["gate"], y, i["dy"], i["h0"], i["dl"], lengths=i["L"], **o)
    ds, dw = hc.hc_rms_norm_backward(a["s"], i["w"], dx.view(B * S, C), ds=i["r"], **o)
    b = hc.xhc_balance_loss(i["score"], i["idx"], B, S, m=m, **o)
    dsc = hc.xhc_balance_loss_backward(i["score"], b["count"], b["tokens"], k, B, S, **o)
    dX, dwr = hc.xhc_router_backward(i["X"], i["wr"], i["score"], dsc, i["dX"], out=torch.empty_like(i["dX"]), **o)
    return [a["y"], a["s"], q["y"].view(torch.uint8), q["scale"], p["y"], p["F_in"], y, last, dx, dg, dh0, ds, dw,
            b["loss"], b["count"], b["tokens"], b["mean_p"], dsc, dX, dwr]


def _same(a, b, what=""):
    for n, (u, v) in enumerate(zip(a, b)):
        assert torch.equal(u, v), f"{what} output {n}"


def test_the_same_every_time():
    note("every call five times: bit-identical")
    i = _inputs(1, S=3000)
    want = _step(i)
    for _ in range(5):
        _same(want, _step(i), "again")


def test_captured_and_replayed():
    note("graph of every call, replayed with new inputs and eager work between")
    i, j = _inputs(2), _inputs(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(i)
    torch.cuda.current_stream().wait_stream(side)
    buf = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in i.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(buf)
    for rep in range(4):
        src = j if rep % 2 else i
        for k, v in src.items():
            if isinstance(v, torch.Tensor):
                buf[k].copy_(v)
        graph.replay()
        want = _step(src)  # eager work of its own between the replays
        torch.cuda.synchronize()
        _same(want, outs, f"replay {rep}")


def test_two_graphs_and_eager_calls_interleaved():
    note("two graphs with their own workspaces, replayed in turn")
    made = []
    for seed in (4, 5):
        i = _inputs(seed, S=900 + seed)
        _step(i)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _step(i)
        made.append((graph, outs, [t.clone() for t in _step(i)], i))  # the graph reads i's arrays
    for _ in range(3):
        for graph, outs, want, _ in made:
            for t in outs:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _ in made:
            _same(want, outs)


def test_two_streams_at_once():
    note("the same calls on two streams at once")
    i, j = _inputs(6, S=4000), _inputs(7, S=3500)
    wi, wj = _step(i), _step(j)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        with torch.cuda.stream(a):
            gi = _step(i)
        with torch.cuda.stream(b):
            gj = _step(j)
        got.append((gi, gj))
    torch.cuda.synchronize()
    for gi, gj in got:
        _same(wi, gi)
        _same(wj, gj)


def test_explicit_stream_keeps_its_workspace():
    note("stream= another stream than the current one, the current one allocating at once")
    i = _inputs(8, S=4000)
    want = _step(i)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = []
    for _ in range(4):
        with torch.cuda.stream(other):
            torch.cuda._sleep(2_000_000)
        got = _step(i, stream=other.cuda_stream)
        # what the current stream allocates now must not be memory the other still works on
        junk += [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (64, 1 << 12, 1 << 16, 1 << 20, 1 << 22)]
        other.synchronize()
        _same(want, got, "explicit stream")
    _same(want, _step(i, stream=0), "default stream")


@pytest.mark.parametrize("S", [1, 100, 129, 700, 1024, 1500, 9000])
def test_scan_state_in_place(S):
    note(f"scan with h_last written over h0, S={S}")
    g = torch.Generator(device="cuda").manual_seed(S)
    B, C = 3, 2050
    x, gate = torch.randn(B, S, C, device="cuda", generator=g), 4 + torch.randn(B, S, C, device="cuda", generator=g)
    h0 = 100 * torch.randn(B, C, device="cuda", generator=g)
    y, last = hc.hc_gated_scan(x, gate, h0)
    for _ in range(5):
        state = h0.clone()
        y2, l2 = hc.hc_gated_scan(x, gate, state, out=(None, state))
        assert l2 is state and torch.equal(y2, y) and torch.equal(state, last)


def test_batches_do_not_touch_each_other():
    note("scan: a sequence alone gives what it gives in a batch")
    g = torch.Generator(device="cuda").manual_seed(9)
    B, S, C = 5, 777, 130
    x = torch.randn(B, S, C, device="cuda", generator=g).bfloat16()
    gate = 2 + torch.randn(B, S, C, device="cuda", generator=g).bfloat16()
    y, last = hc.hc_gated_scan(x, gate)
    for b in range(B):
        yb, lb = hc.hc_gated_scan(x[b:b + 1].contiguous(), gate[b:b + 1].contiguous())
        assert torch.equal(yb[0], y[b]) and torch.equal(lb[0], last[b])


@pytest.mark.slow
def test_offsets_past_32_bits():
    note("norm, scan and router backward on arrays of more than 2^31 elements")
    g = torch.Generator(device="cuda").manual_seed(10)
    T, C = 140_000, 16384  # 2.3e9 elements
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    r = hc.hc_rms_norm(x, quant=torch.float8_e4m3fn, group=128)
    tail = hc.hc_rms_norm(x[-5:].contiguous(), quant=torch.float8_e4m3fn, group=128)
    assert torch.equal(r["y"][-5:].view(torch.uint8), tail["y"].view(torch.uint8))
    assert torch.equal(r["scale"][-5:], tail["scale"])
    del r
    dx, _ = hc.hc_rms_norm_backward(x, None, x, want_dweight=False)
    tx, _ = hc.hc_rms_norm_backward(x[-5:].contiguous(), None, x[-5:].contiguous(), want_dweight=False)
    assert torch.equal(dx[-5:], tx)
    B, S = 2, T // 2
    y, last = hc.hc_gated_scan(x.view(B, S, C), dx.view(B, S, C))
    yt, lt = hc.hc_gated_scan(x.view(B, S, C)[1:, :, -64:].contiguous(), dx.view(B, S, C)[1:, :, -64:].contiguous())
    assert torch.equal(y[1, :, -64:], yt[0]) and torch.equal(last[1, -64:], lt[0])
    del y, last, dx
    N, Cn = 16, 4096
    Tn = T * C // (N * Cn)  # 35,000 tokens
    X = x.view(-1)[:Tn * N * Cn].view(Tn, N, Cn)
    ds = torch.randn(Tn, 14, device="cuda", generator=g)
    ds[:-64] = 0  # only the last 64 tokens take part
    score = torch.sigmoid(torch.randn(Tn, 14, device="cuda", generator=g))
    w = 0.01 * torch.randn(N * Cn, 14, device="cuda", generator=g)
    out, dw = hc.xhc_router_backward(X, w, score, ds, X, out=torch.empty_like(X))
    o2, dw2 = hc.xhc_router_backward(X[-64:].contiguous(), w, score[-64:].contiguous(), ds[-64:].contiguous(),
                                     X[-64:].clone())
    torch.cuda.synchronize()
    assert torch.equal(out[-64:], o2)
    assert torch.allclose(dw, dw2, rtol=0, atol=float(dw2.abs().max()) * 1e-6)
    assert torch.equal(out[:100], X[:100])


def test_other_device_than_the_current_one():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    i = _inputs(11)
    j = {k: v.to("cuda:1") if isinstance(v, torch.Tensor) else v for k, v in i.items()}
    a = hc.hc_rms_norm(j["x"], j["w"], residual=j["r"])
    assert torch.equal(a["y"].to("cuda:0"), hc.hc_rms_norm(i["x"], i["w"], residual=i["r"])["y"])


# ------------------------------------------------------------------ together


def test_static_mhc_around_a_scan_block_forward_and_backward():
    """A static-mHC sublayer whose function is norm, two projections and the gated scan: the library's
    calls against the same step written in float64 torch with autograd. Every stored bfloat16 value rounds
    by at most 2^-8; five are chained forward (F_in, y, two projections, h) and as many backward, so the
    gradients agree to a few per cent of their norm (12 roundings of 2^-8 in a row are 4.7 %)."""
    note("static mHC around norm + scan, forward and backward")
    B, S, n, C = 2, 150, 4, 64
    T = B * S
    g = torch.Generator().manual_seed(12)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    X64 = rn(T, n, C).bfloat16().double()
    w64, Wx, Wg = 1 + 0.1 * rn(C), (rn(C, C) / 8).bfloat16().double(), (rn(C, C) / 8).bfloat16().double()
    logits, dN = rn(n * n + 2 * n).float(), rn(T, n, C).bfloat16()

    # the library
    X = X64.bfloat16().cuda()
    h_pre, h_post, h_res = hc.hc_static_maps(logits.cuda(), n)
    F_in = hc.hc_static_pre(X, h_pre)
    wd, Wxd, Wgd = w64.float().cuda(), Wx.bfloat16().cuda(), Wg.bfloat16().cuda()
    y = hc.hc_rms_norm(F_in, wd)["y"]
    xs, gs = (y @ Wxd).view(B, S, C), (y @ Wgd).view(B, S, C)
    hs, _ = hc.hc_gated_scan(xs, gs)
    Xn = hc.hc_static_post(X, h_res, h_post, hs.view(T, C))
    fused = hc.hc_pre_norm(X, h_pre.expand(T, n).contiguous(), wd)
    # the fused call forms y from F_in before its rounding: two roundings of 2^-8 apart at most
    assert torch.allclose(fused["y"].float(), y.float(), rtol=2.0 ** -6, atol=1e-6)
    dNd = dN.cuda()
    dF = torch.einsum("i,tic->tc", h_post, dNd.float()).bfloat16()
    dxs, dgs, _ = hc.hc_gated_scan_backward(xs, gs, hs, dF.view(B, S, C))
    dy = (dxs.view(T, C).float() @ Wxd.float().t() + dgs.view(T, C).float() @ Wgd.float().t()).bfloat16()
    dF_in, dw = hc.hc_rms_norm_backward(F_in, wd, dy)

    # float64 with autograd
    Xr, wr = X64.clone().requires_grad_(), w64.clone().requires_grad_()
    hp, hq, hr = h_pre.cpu().double(), h_post.cpu().double(), h_res.cpu().double()
    F = torch.einsum("i,tic->tc", hp, Xr)
    F.retain_grad()
    yr = F / (F.square().mean(1, keepdim=True) + 1e-6).sqrt() * wr
    xr, gr = (yr @ Wx).view(B, S, C), torch.sigmoid((yr @ Wg).view(B, S, C))
    h, hsr = torch.zeros(B, C, dtype=torch.float64), []
    for t in range(S):
        h = gr[:, t] * h + (1 - gr[:, t]) * xr[:, t]
        hsr.append(h)
    hsr = torch.stack(hsr, 1).view(T, C)
    Xnr = torch.einsum("ij,tjc->tic", hr, Xr) + hq[None, :, None] * hsr[:, None]
    Xnr.backward(dN.double())
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(Xn, Xnr.detach()) < 0.02
    assert rel(hs.view(T, C), hsr.detach()) < 0.03
    assert rel(dF_in, F.grad) < 0.05
    assert rel(dw, wr.grad) < 0.05


def test_routed_step_with_balance_loss_trains_its_router():
    """A routed xHC sublayer with the balance loss: the gradients that the loss sends through the scores
    to w_router and the state, against float64 autograd of the loss with the counts held (they are exact:
    the routing itself is the library's). float32 scores and a bfloat16 dX: 2^-8 on dX, 1e-4 on dw."""
    note("xhc_pre, norm, scan, augment, route, balance loss and the router's backward")
    B, S, N, k, m, C = 2, 60, 8, 4, 2, 64
    T, E = B * S, N - m
    g = torch.Generator().manual_seed(13)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    X = rn(T, N, C).bfloat16().cuda()
    wr = (rn(N * C, E) * 2 / (N * C) ** 0.5).cuda()
    pre = hc.xhc_pre(X, 0.01 * rn(N * C, N).cuda(), rn(N).cuda(), 0.01, wr, k, m)
    y = hc.hc_rms_norm(pre["F_in"], eps=1e-6)["y"]
    hs, _ = hc.hc_gated_scan(y.view(B, S, C), (2 + rn(B, S, C)).bfloat16().cuda())
    V = hc.xhc_augment(hs.view(T, C), 0.3 * rn(C * 24).cuda(), (4, 8, 12), B, S)
    X0 = X.clone()
    hc.xhc_route(X, V, 0.01 * rn(k * C, k * 4 + k * k).cuda(), rn(k * 4 + k * k).cuda(), 0.01, 0.01, k=k, m=m,
                 idx=pre["idx"])
    bal = hc.xhc_balance_loss(pre["score"], pre["idx"], B, S, m=m, coef=0.5)
    ds = hc.xhc_balance_loss_backward(pre["score"], bal["count"], bal["tokens"], k, B, S, coef=0.5)
    dX0 = (0.001 * rn(T, N, C)).bfloat16().cuda()
    dX, dw = hc.xhc_router_backward(X0, wr, pre["score"], ds, dX0, out=torch.empty_like(dX0))
    torch.cuda.synchronize()

    Xr, Wr = X0.cpu().double().requires_grad_(), wr.cpu().double().requires_grad_()
    x = Xr.view(T, N * C)
    score = torch.sigmoid((x @ Wr) / x.square().mean(1, keepdim=True).sqrt())
    p = (score / score.sum(1, keepdim=True)).view(B, S, E)
    idx = pre["idx"].cpu().view(B, S * k).long()
    count = torch.stack([torch.bincount(i, minlength=N) for i in idx]).double()
    f = count[:, m:] * E / ((k - m) * S)
    loss = 0.5 * (f * p.mean(1)).sum() / B
    loss.backward()
    assert torch.equal(bal["count"].cpu().long(), count.long())
    assert abs(float(bal["loss"]) - float(loss)) < 1e-5 * float(loss)
    assert int(bal["count"].sum()) == T * k and bool((bal["count"][:, :m] == S).all())
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(dw, Wr.grad) < 1e-4
    want = dX0.cpu().double() + Xr.grad
    assert bool(((dX.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * Xr.grad.abs().max()).all())
    # a step against the gradient lowers the loss to first order
    step = 1e-3 / float(Wr.grad.norm())
    with torch.no_grad():
        s2 = torch.sigmoid((x @ (Wr - step * dw.cpu().double())) / x.square().mean(1, keepdim=True).sqrt())
        l2 = 0.5 * (f * (s2 / s2.sum(1, keepdim=True)).view(B, S, E).mean(1)).sum() / B
    slope = float((Wr.grad * dw.cpu().double()).sum()) * step
    assert abs(float(loss - l2) - slope) < 0.05 * slope


def _raises(exc, fn, *a, **k):
    with pytest.raises(exc):
        fn(*a, **k)


def test_binding_refuses_wrong_arguments():
    note("binding validation: norm, scan and router calls")
    i = _inputs(14, S=5, C=64)
    x, w, X = i["x"], i["w"], i["X"]
    e4 = torch.float8_e4m3fn
    _raises(ValueError, hc.hc_rms_norm, x.view(2, 5, 64), w)
    _raises(ValueError, hc.hc_rms_norm, x, w[:-1])
    _raises(TypeError, hc.hc_rms_norm, x, w.bfloat16())
    _raises(TypeError, hc.hc_rms_norm, x.half(), w)
    _raises(ValueError, hc.hc_rms_norm, x.t(), None)
    _raises(ValueError, hc.hc_rms_norm, x, w, residual=i["r"][:4])
    _raises(TypeError, hc.hc_rms_norm, x, w, residual=i["r"].float())
    _raises(ValueError, hc.hc_rms_norm, x, w, s_out=torch.empty_like(x))  # no residual
    _raises(ValueError, hc.hc_rms_norm, x, w, group=32)  # no 8-bit output
    _raises(ValueError, hc.hc_rms_norm, x, w, quant=e4, group=48)
    _raises(TypeError, hc.hc_rms_norm, x, w, quant=torch.float8_e5m2)
    _raises(ValueError, hc.hc_rms_norm, x, w, quant=e4, out=(None, torch.empty(10, 2, device="cuda")))
    _raises(TypeError, hc.hc_rms_norm, x, w, quant=e4, out=(torch.empty_like(x), None))
    _raises(hc.HCError, hc.hc_rms_norm, x, w, -1.0)
    _raises(hc.HCError, hc.hc_rms_norm, x, w, out=(x, None))  # y over x
    _raises(hc.HCError, hc.hc_rms_norm, torch.zeros(1, 16392, device="cuda"))
    _raises(ValueError, hc.hc_pre_norm, X, i["h"][:, :4].contiguous(), w)
    _raises(ValueError, hc.hc_pre_norm, X, i["h"], w, F_in_out=torch.empty(5, 64, dtype=x.dtype, device="cuda"))
    _raises(ValueError, hc.hc_rms_norm_backward, x, w, x[:3])
    _raises(ValueError, hc.hc_rms_norm_backward, x, w, x, ds=x[:, :32].contiguous())
    _raises(hc.HCError, hc.hc_rms_norm_backward, x, w, x, out=(x, None))
    xs = x.view(2, 5, 64)
    _raises(ValueError, hc.hc_gated_scan, x, i["gate"])
    _raises(ValueError, hc.hc_gated_scan, xs, i["gate"][:, :4].contiguous())
    _raises(TypeError, hc.hc_gated_scan, xs, i["gate"].float())
    _raises(ValueError, hc.hc_gated_scan, xs, i["gate"], i["h0"][:1])
    _raises(TypeError, hc.hc_gated_scan, xs, i["gate"], lengths=i["L"].long())
    _raises(ValueError, hc.hc_gated_scan, xs, i["gate"], lengths=i["L"][:1])
    _raises(hc.HCError, hc.hc_gated_scan, xs, i["gate"], out=(xs, None))
    _raises(ValueError, hc.hc_gated_scan_backward, xs, i["gate"], xs, i["dy"][:1])
    _raises(hc.HCError, hc.hc_gated_scan_backward, xs, i["gate"], xs, i["dy"], out=(i["dy"], None, None))
    sc, idx = i["score"], i["idx"]
    _raises(ValueError, hc.xhc_balance_loss, sc, idx, 2, 6)
    _raises(ValueError, hc.xhc_balance_loss, sc, idx[:4], 2, 5)
    _raises(TypeError, hc.xhc_balance_loss, sc, idx.long(), 2, 5)
    _raises(ValueError, hc.xhc_balance_loss, sc, idx, 2, 5, mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    _raises(hc.HCError, hc.xhc_balance_loss, sc, idx[:, :2].contiguous(), 2, 5)  # k = m: nothing is chosen
    b = hc.xhc_balance_loss(sc, idx, 2, 5)
    _raises(ValueError, hc.xhc_balance_loss_backward, sc, b["count"][:1], b["tokens"], 4, 2, 5)
    _raises(ValueError, hc.xhc_balance_loss_backward, sc, b["count"], b["tokens"], 4, 2, 5,
            dloss=torch.ones(2, device="cuda"))
    ds = torch.zeros_like(sc)
    _raises(ValueError, hc.xhc_router_backward, X, i["wr"][:-1], sc, ds, i["dX"])
    _raises(ValueError, hc.xhc_router_backward, X, i["wr"], sc, ds[:3], i["dX"])
    _raises(TypeError, hc.xhc_router_backward, X.float(), i["wr"], sc, ds, i["dX"].float())
    _raises(hc.HCError, hc.xhc_router_backward, X, i["wr"], sc, ds, X)  # in place on the state itself
    assert torch.isfinite(hc.xhc_balance_loss(sc, idx, 2, 5)["loss"])  # a valid call after the refusals


@pytest.mark.parametrize("default", ["float64", "bfloat16"])
def test_program_with_another_default_type(default):
    """What a call allocates is float32 where the library writes float32."""
    i = _inputs(23)
    want = _step(i)
    before = torch.get_default_dtype()
    try:
        torch.set_default_dtype(getattr(torch, default))
        got = _step(i)
    finally:
        torch.set_default_dtype(before)
    assert [t.dtype for t in got] == [t.dtype for t in want]
    _same(got, want, f"default type {default}")
