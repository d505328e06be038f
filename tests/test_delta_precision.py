"""The tolerances of the gated delta rule's precision tests, on the CPU: the chunked form is the recurrence, and
the losses that those tests are there for lie outside the tolerances."""
import numpy as np
import pytest

import delta_precision as D
from oracle import sublayer_ops as R


def _head(ins, h=0):
    q, k, v, g, beta, M = ins[:6]
    return q[0, :, 0], k[0, :, 0], v[0, :, h], g[0, :, h], beta[0, :, h], M[0, h]


@pytest.mark.parametrize("segment", [None, 256])
def test_chunked_is_the_recurrence(segment):
    ins = D.inputs(1, 700, 1, 1, 32, 24, "f32", 1)
    o, M = R.gated_delta(*ins[:6])
    oc, Mc = D.chunked(*_head(ins), 32 ** -0.5, segment=segment)
    assert D.rel(oc, o[0, :, 0]) < 1e-12 and D.rel(Mc, M[0, 0]) < 1e-12


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(300, 64, 48), (200, 128, 64)])
def test_factors_in_two_parts_are_told(dt, size):
    """Three parts lie within the tolerances, two outside, in both stream types."""
    S, Dk, Dv = size
    ins = D.inputs(1, S, 1, 1, Dk, Dv, dt, S)
    o, M = R.gated_delta(*ins[:6])
    o, M = o[0, :, 0], M[0, 0]
    o3, M3 = D.chunked(*_head(ins), Dk ** -0.5, held=3)
    o2, M2 = D.chunked(*_head(ins), Dk ** -0.5, held=2)
    assert D.rel(o3, o) < D.OUT / 8 and D.rel(M3, M) < D.STATE / 8
    assert D.rel(o2, o) > D.OUT and D.rel(M2, M) > D.STATE


@pytest.mark.parametrize("n", [300, 12000, 1 << 18, 1 << 20])
def test_a_bfloat16_result_tells_an_error_before_its_rounding(n):
    """Errors of 2^-20 stay inside the tolerance of a rounded result, of 2^-18.5 do not where there are many."""
    rng = np.random.default_rng(n)
    y = rng.normal(size=n)
    off = lambda e: D.rel(D.bf16(y + e * rng.normal(size=n)), D.bf16(y))  # noqa: E731
    assert off(2.0 ** -20) < D.half(D.bf16(y))
    assert n < 10000 or D.half(D.bf16(y)) < off(2.0 ** (-18.5 if n >= 1 << 18 else -13))


@pytest.mark.parametrize("size", [(1100, 128, 24, 320), (2100, 64, 32, 320)])
def test_segments_need_their_maps(size):
    """The inputs of the segments' tests carry the first state to the last: without the maps the result is another."""
    S, Dk, Dv, segment = size
    head = _head(D.inputs(1, S, 1, 1, Dk, Dv, "f32", S, slow=1e-4))
    o, M = D.chunked(*head, Dk ** -0.5)
    os, Ms = D.chunked(*head, Dk ** -0.5, segment=segment)
    oz, Mz = D.chunked(*head, Dk ** -0.5, segment=segment, maps="zero")
    grow = D.joins(S)
    assert D.rel(os, o) < D.OUT * grow / 8 and D.rel(Ms, M) < D.STATE * grow / 8
    assert D.rel(oz, o) > 0.1 and D.rel(Mz, M) > 0.1


def test_maps_in_two_parts_are_told():
    """Over many segments, what two parts leave of the maps and the joined states adds up."""
    S, Dk, Dv = 8192, 128, 8
    head = _head(D.inputs(1, S, 1, 1, Dk, Dv, "f32", 5, slow=1e-5))
    o, M = D.chunked(*head, Dk ** -0.5)
    two, M2 = D.chunked(*head, Dk ** -0.5, segment=256, map_parts=2)
    three, M3 = D.chunked(*head, Dk ** -0.5, segment=256, map_parts=3)
    grow = D.joins(S)
    assert D.rel(M3, M) < D.STATE * grow / 8 and D.rel(three, o) < D.OUT * grow / 8
    assert D.rel(M2, M) > 2 * D.STATE * grow and D.rel(two, o) > D.OUT * grow
