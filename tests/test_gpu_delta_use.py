"""The layer norm and gated delta rule calls as a program uses them: captured and replayed, on other
streams, several at once, with the same results every time, on arrays past 2^31 elements, and
together with the stream mixing in a forward and backward step."""
import pytest

from hc_testutil import have_gpu, note

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc


def _inputs(seed, B=2, S=1100, C=512, Hk=2, Hv=4, Dk=64, Dv=96):
    """S of 1,024 and more at so few heads: a sequence walked in segments."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1).bfloat16()  # noqa: E731
    T = B * S
    return dict(x=rn(T, C).bfloat16(), r=rn(T, C).bfloat16(), w=1 + 0.1 * rn(C), b=0.1 * rn(C), X=rn(T, 4, C).bfloat16(),
                h=torch.sigmoid(rn(T, 4)), q=unit(rn(B, S, Hk, Dk)), k=unit(rn(B, S, Hk, Dk)),
                v=rn(B, S, Hv, Dv).bfloat16(), g=-torch.exp(rn(B, S, Hv) - 3), be=torch.sigmoid(rn(B, S, Hv)),
                M=0.3 * rn(B, Hv, Dk, Dv), do=rn(B, S, Hv, Dv).bfloat16(), dM=0.3 * rn(B, Hv, Dk, Dv),
                L=torch.tensor([S, S // 3] + [S] * (B - 2), dtype=torch.int32, device="cuda"))


def _step(i, stream=None):
    """Every new call once, the delta rule also for single tokens; all outputs."""
    o = {"stream": stream}
    a = hc.hc_layer_norm(i["x"], i["w"], i["b"], residual=i["r"], **o)
    e = hc.hc_layer_norm(i["x"], i["w"], i["b"], residual=i["r"], quant=torch.float8_e4m3fn, group=128, **o)
    p = hc.hc_pre_layer_norm(i["X"], i["h"], i["w"], i["b"], **o)
    ln = hc.hc_layer_norm_backward(a["s"], i["w"], p["y"], ds=i["r"], **o)
    d = [i[n] for n in ("q", "k", "v", "g", "be")]
    y, last = hc.hc_gated_delta(*d, i["M"], lengths=i["L"], out=(torch.zeros_like(i["v"]), None), **o)
    one = [t[:, :1].contiguous() for t in d]
    y1, last1 = hc.hc_gated_delta(*one, last, **o)
    back = hc.hc_gated_delta_backward(*d, i["do"], i["M"], i["dM"], lengths=i["L"], **o)
    return [a["y"], a["s"], e["y"].view(torch.uint8), e["scale"], p["y"], p["F_in"], *ln, y, last, y1, last1, *back]


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
    buf = {k: v.clone() for k, v in i.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(buf)
    for rep in range(4):
        src = j if rep % 2 else i
        for k, v in src.items():
            buf[k].copy_(v)
        graph.replay()
        want = _step(src)  # eager work of its own between the replays
        torch.cuda.synchronize()
        _same(want, outs, f"replay {rep}")


def test_two_graphs_and_eager_calls_interleaved():
    note("two graphs with their own workspaces, replayed in turn")
    made = []
    for seed in (4, 5):
        i = _inputs(seed, S=900 + 100 * seed)
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
    for _ in range(4):
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
    d = [i[n] for n in ("q", "k", "v", "g", "be")]
    for _ in range(4):
        with torch.cuda.stream(other):
            torch.cuda._sleep(2_000_000)
        o = {"stream": other.cuda_stream}
        y, last = hc.hc_gated_delta(*d, i["M"], **o)
        back = hc.hc_gated_delta_backward(*d, i["do"], i["M"], i["dM"], lengths=i["L"], **o)
        ln = hc.hc_layer_norm_backward(i["x"], i["w"], i["r"], **o)
        # what the current stream allocates now must not be memory the other still works on
        junk += [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (64, 1 << 12, 1 << 16, 1 << 20, 1 << 22)]
        other.synchronize()
        _same(want[-6:], back, "backward")
        _same(hc.hc_layer_norm_backward(i["x"], i["w"], i["r"]), ln, "layer norm")
        _same(hc.hc_gated_delta(*d, i["M"]), (y, last), "forward")


@pytest.mark.parametrize("S", [1, 8, 9, 64, 700, 2000])
def test_state_in_place(S):
    note(f"last state written over the given one, S={S}")
    i = _inputs(20 + S, B=3, S=S)
    d = [i[n] for n in ("q", "k", "v", "g", "be")]
    y, last = hc.hc_gated_delta(*d, i["M"], lengths=i["L"])
    for _ in range(3):
        state = i["M"].clone()
        y2, l2 = hc.hc_gated_delta(*d, state, lengths=i["L"], out=(None, state))
        assert l2 is state and torch.equal(y2, y) and torch.equal(state, last)


def test_state_in_place_beside_other_work():
    """A long sequence's segments are walked at once, in whatever order the workgroups start: the first must
    not read the state that the last one has written over it."""
    note("last state written over the given one, five streams at once")
    runs = []
    for s in range(5):
        i = _inputs(40 + s, B=1, S=4000, Hk=4, Hv=16, Dk=128, Dv=128)
        d = [i[n] for n in ("q", "k", "v", "g", "be")]
        runs.append((d, i["M"], hc.hc_gated_delta(*d, i["M"]), [i["M"].clone() for _ in range(4)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [(hc.hc_gated_delta(*d, state, out=(None, state), stream=st.cuda_stream), want)
           for k in range(4) for d, _, want, states, st in runs for state in (states[k],)]
    torch.cuda.synchronize()
    for g, want in got:
        _same(want, g)


def test_batches_do_not_touch_each_other():
    note("a sequence alone gives what it gives in a batch, forward and backward")
    i = _inputs(9, B=4, S=500)
    d = [i[n] for n in ("q", "k", "v", "g", "be")]
    y, last = hc.hc_gated_delta(*d, i["M"])
    back = hc.hc_gated_delta_backward(*d, i["do"], i["M"], i["dM"])
    for b in range(4):
        e = [t[b:b + 1].contiguous() for t in d]
        M, do, dM = (i[n][b:b + 1].contiguous() for n in ("M", "do", "dM"))
        yb, lb = hc.hc_gated_delta(*e, M)
        assert torch.equal(yb[0], y[b]) and torch.equal(lb[0], last[b])
        for x, xb in zip(back, hc.hc_gated_delta_backward(*e, do, M, dM)):
            assert torch.equal(x[b], xb[0])


def test_the_same_array_twice():
    note("q and k, or do and v, may be one array")
    i = _inputs(10, S=130)
    d = [i["k"], i["k"], i["v"], i["g"], i["be"]]
    e = [i["k"].clone(), *d[1:]]
    _same(hc.hc_gated_delta(*d, i["M"]), hc.hc_gated_delta(*e, i["M"]))
    _same(hc.hc_gated_delta_backward(*d, i["v"], i["M"], i["M"]),
          hc.hc_gated_delta_backward(*e, i["v"].clone(), i["M"], i["M"].clone()))


@pytest.mark.slow
def test_offsets_past_32_bits():
    note("norm and delta rule on arrays of more than 2^31 elements")
    g = torch.Generator(device="cuda").manual_seed(10)
    T, C = 140_000, 16384  # 2.3e9 elements
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    t = x[-5:].contiguous()
    assert torch.equal(hc.hc_layer_norm(x)["y"][-5:], hc.hc_layer_norm(t)["y"])
    dx = hc.hc_layer_norm_backward(x, None, x, want_dweight=False)[0]
    assert torch.equal(dx[-5:], hc.hc_layer_norm_backward(t, None, t, want_dweight=False)[0])
    del dx
    # one sequence of 64 value heads of 256: the last head alone, and the backward of both
    S, Hv, Dk, Dv = 140_000, 64, 32, 256
    v = x.view(1, S, Hv, Dv)
    q = torch.nn.functional.normalize(torch.randn(1, S, 1, Dk, device="cuda", generator=g), dim=-1).bfloat16()
    gd = torch.full((1, S, Hv), -0.05, device="cuda")
    be = torch.rand(1, S, Hv, device="cuda", generator=g)
    e = [q, q, v[:, :, -1:].contiguous(), gd[..., -1:].contiguous(), be[..., -1:].contiguous()]
    y, last = hc.hc_gated_delta(q, q, v, gd, be)
    yt, lt = hc.hc_gated_delta(*e)
    # the segments' lengths depend on the number of heads: the same sums in another order, 2^-15 of a state of
    # norm at most |v| / (1 - e^-0.05), and a rounding of 2^-8 to bfloat16 in each
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
    assert rel(y[0, :, -1], yt[0, :, 0]) < 2 * 2.0 ** -8 and rel(last[0, -1], lt[0, 0]) < 21 * 2.0 ** -15
    del y
    back = hc.hc_gated_delta_backward(q, q, v, gd, be, v)
    bt = hc.hc_gated_delta_backward(*e, e[2])
    assert rel(back[2][0, :, -1], bt[2][0, :, 0]) < 2 * 2.0 ** -8
    assert rel(back[4][0, :, -1], bt[4][0, :, 0]) < 21 * 2.0 ** -8
    del back
    # states of 2.3e9 floats, one token each
    del x, v
    B, H = 2_200, 16
    M = torch.empty(B, H, 256, 256, device="cuda").normal_(generator=g)
    a = [torch.randn(B, 1, H, 256, device="cuda", generator=g) / 16 for _ in range(3)]
    s = [-torch.rand(B, 1, H, device="cuda", generator=g), torch.rand(B, 1, H, device="cuda", generator=g)]
    y, last = hc.hc_gated_delta(*a, *s, M)
    yt, lt = hc.hc_gated_delta(*(t[-3:].contiguous() for t in (*a, *s)), M[-3:].contiguous())
    assert torch.equal(y[-3:], yt) and torch.equal(last[-3:], lt)


def test_other_device_than_the_current_one():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    i = _inputs(11)
    j = {k: v.to("cuda:1") for k, v in i.items()}
    _same([t.cpu() for t in _step(i)], [t.cpu() for t in _step(j)])


@pytest.mark.parametrize("default", ["float64", "bfloat16"])
def test_program_with_another_default_type(default):
    """What a call allocates is float32 where the library writes float32."""
    i = _inputs(23, S=150)
    want = _step(i)
    before = torch.get_default_dtype()
    try:
        torch.set_default_dtype(getattr(torch, default))
        got = _step(i)
    finally:
        torch.set_default_dtype(before)
    assert [t.dtype for t in got] == [t.dtype for t in want]
    _same(got, want, f"default type {default}")


def test_static_mhc_around_a_delta_block_forward_and_backward():
    """A static-mHC sublayer whose function is the layer norm, projections, the root-mean-square norm of each
    head's q and k to unit length, and the gated delta rule: the library's calls against the same step in
    float64 torch with autograd. Every stored bfloat16 value rounds by at most 2^-8; six are chained forward
    (F_in, y, projections, q and k, o, X') and as many backward, so gradients agree to 12 roundings of 2^-8 in
    a row, 4.7 %, of their norm."""
    note("static mHC around layer norm + gated delta rule, forward and backward")
    B, S, n, C, Hk, Hv, Dk, Dv = 2, 150, 4, 96, 2, 4, 16, 24
    T = B * S
    rng = torch.Generator().manual_seed(12)
    rn = lambda *s: torch.randn(*s, generator=rng, dtype=torch.float64)  # noqa: E731
    X64, dN = rn(T, n, C).bfloat16().double(), rn(T, n, C).bfloat16()
    w64, b64 = 1 + 0.1 * rn(C), 0.1 * rn(C)
    Wq, Wk, Wv = ((rn(C, w) / C ** 0.5).bfloat16().double() for w in (Hk * Dk, Hk * Dk, C))
    assert Hv * Dv == C
    logits, gd, be = rn(n * n + 2 * n).float(), -torch.exp(rn(B, S, Hv) - 2).float(), torch.sigmoid(rn(B, S, Hv)).float()

    # the library
    X, wd, bd = X64.bfloat16().cuda(), w64.float().cuda(), b64.float().cuda()
    h_pre, h_post, h_res = hc.hc_static_maps(logits.cuda(), n)
    f = hc.hc_pre_layer_norm(X, h_pre.expand(T, n).contiguous(), wd, bd, 1e-6)
    F_in, y = f["F_in"], f["y"]
    Wqd, Wkd, Wvd = (W.bfloat16().cuda() for W in (Wq, Wk, Wv))
    one = torch.full((Dk,), Dk ** -0.5, device="cuda")  # a root mean square of Dk^-1/2 is a norm of 1
    qr, kr = ((y @ W).view(T * Hk, Dk) for W in (Wqd, Wkd))
    q, k = (hc.hc_rms_norm(t, one)["y"].view(B, S, Hk, Dk) for t in (qr, kr))
    v = (y @ Wvd).view(B, S, Hv, Dv)
    o, last = hc.hc_gated_delta(q, k, v, gd.cuda(), be.cuda())
    Xn = hc.hc_static_post(X, h_res, h_post, o.view(T, C))
    dF = torch.einsum("i,tic->tc", h_post, dN.cuda().float()).bfloat16()
    dq, dk, dv, dg, db, _ = hc.hc_gated_delta_backward(q, k, v, gd.cuda(), be.cuda(), dF.view(B, S, Hv, Dv))
    dqr, dkr = (hc.hc_rms_norm_backward(r, one, d.view(T * Hk, Dk), want_dweight=False)[0].view(T, Hk * Dk)
                for r, d in ((qr, dq), (kr, dk)))
    dy = (dqr.float() @ Wqd.float().t() + dkr.float() @ Wkd.float().t() + dv.view(T, C).float() @ Wvd.float().t()).bfloat16()
    dF_in, dw, dbias = hc.hc_layer_norm_backward(F_in, wd, dy, 1e-6)

    # float64 with autograd
    Xr, wr, br = (t.clone().requires_grad_() for t in (X64, w64, b64))
    gr, ber = gd.double().requires_grad_(), be.double().requires_grad_()
    F = torch.einsum("i,tic->tc", h_pre.cpu().double(), Xr)
    F.retain_grad()
    c = F - F.mean(1, keepdim=True)
    yr = c / (c.square().mean(1, keepdim=True) + 1e-6).sqrt() * wr + br
    unit = lambda t: t / (t.square().sum(-1, keepdim=True) + Dk * 1e-6).sqrt()  # noqa: E731
    q6, k6 = (unit((yr @ W).view(B, S, Hk, Dk)).repeat_interleave(Hv // Hk, 2) for W in (Wq, Wk))
    v6 = (yr @ Wv).view(B, S, Hv, Dv)
    M, os = torch.zeros(B, Hv, Dk, Dv, dtype=torch.float64), []
    for t in range(S):
        M = M * gr[:, t, :, None, None].exp()
        z = v6[:, t] - (M * k6[:, t, :, :, None]).sum(2)
        M = M + ber[:, t, :, None, None] * k6[:, t, :, :, None] * z[:, :, None]
        os.append(Dk ** -0.5 * (M * q6[:, t, :, :, None]).sum(2))
    or_ = torch.stack(os, 1).view(T, C)
    Xnr = torch.einsum("ij,tjc->tic", h_res.cpu().double(), Xr) + h_post.cpu().double()[None, :, None] * or_[:, None]
    Xnr.backward(dN.double())
    rel = lambda a, b: float((a.double().cpu() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    assert rel(Xn, Xnr) < 0.02
    assert rel(o.view(T, C), or_) < 0.03
    assert rel(last, M) < 0.03
    for name, a, b in (("F_in", dF_in, F.grad), ("w", dw, wr.grad), ("b", dbias, br.grad), ("g", dg, gr.grad),
                       ("beta", db, ber.grad)):
        assert rel(a, b) < 0.05, name
