"""The norm and the scan at the edges of what their definitions allow: padded batches whose output
the call allocates."""
import pytest

from hc_testutil import have_gpu, note
from test_gpu_sublayer import _dt

pytestmark = pytest.mark.gpu

if have_gpu():
    import torch
    import stream_residual_mixing_amd as hc


# ------------------------------------------------- padding of an allocated y


def _dirty(shape, dtype):
    """Leaves NaN in the allocator's free memory of this size."""
    junk = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("S", [1, 20, 100, 600])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_padding_of_an_allocated_output_is_zero(S, dt):
    note(f"hc_gated_scan with lengths and no out, S={S} {dt}")
    B, C = 4, 512
    x, g = (torch.randn(B, S, C, device="cuda").to(_dt(dt)) for _ in range(2))
    L = torch.tensor([S, S // 2, 0, -3], dtype=torch.int32, device="cuda")
    want, last = hc.hc_gated_scan(x, g, lengths=L, out=(torch.zeros_like(x), None))
    for out in (None, (None, None), (None, torch.empty(B, C, device="cuda"))):
        _dirty((B, S, C), x.dtype)
        y, l2 = hc.hc_gated_scan(x, g, lengths=L, out=out)
        assert torch.equal(y, want) and torch.equal(l2, last)
    # what a following norm makes of it: padded rows with dy = 0 add nothing to the weight's gradient
    _dirty((B, S, C), x.dtype)
    y, _ = hc.hc_gated_scan(x, g, lengths=L)
    dy = torch.ones_like(y)
    dy[torch.arange(S, device="cuda")[None] >= L[:, None]] = 0
    dx, dw = hc.hc_rms_norm_backward(y.view(B * S, C), None, dy.view(B * S, C))
    assert torch.isfinite(dw).all() and torch.isfinite(dx).all()


def test_scan_padding_of_an_allocated_output_in_a_graph():
    note("hc_gated_scan with lengths and no out, captured and replayed")
    B, S, C = 3, 200, 256
    x, g = (torch.randn(B, S, C, device="cuda").bfloat16() for _ in range(2))
    L = torch.tensor([S, 7, 0], dtype=torch.int32, device="cuda")
    hc.hc_gated_scan(x, g, lengths=L)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = hc.hc_gated_scan(x, g, lengths=L)
    for lens in ([S, 7, 0], [3, S, 150], [0, 0, 0]):
        L.copy_(torch.tensor(lens, dtype=torch.int32))
        y.fill_(float("nan"))
        graph.replay()
        want, wl = hc.hc_gated_scan(x, g, lengths=L, out=(torch.zeros_like(x), None))
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(last, wl)
