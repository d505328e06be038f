"""Which calls of the gated delta rule walk their sequences in segments, by their workspace (CPU)."""
import pytest


@pytest.fixture(scope="module")
def L():
    import stream_residual_mixing_amd as m

    return m.lib()


RECORD = 3 * 64 * 4 + 2 * 6 * 64 * 8 * 4  # a chunk's decays and betas, T and P, float32


@pytest.mark.parametrize("B,S,H,D,cut", [
    (1, 1024, 16, 128, True), (1, 960, 16, 128, False), (1, 1024, 32, 128, True), (1, 1024, 64, 128, False),
    (1, 2048, 64, 128, True), (1, 1024, 16, 256, True), (1, 2048, 24, 256, False), (1, 4096, 24, 256, True),
    (1, 8192, 32, 256, False), (2, 2048, 64, 128, False), (8, 1024, 16, 128, False)])
def test_few_heads_and_long_sequences_are_cut(L, B, S, H, D, cut):
    """As measured where the rule stands: eight segments and more that fill the device pay from 1,024 tokens on, four
    to seven from 2,048, of 256 keys five to seven from 4,096."""
    need = L.hc_gated_delta_workspace_bytes(B, S, H, H, D, D, 1)
    records = B * H * (S // 64) * RECORD
    assert (need > records) == cut, (need, records)
    assert cut or need == records


def test_a_call_without_heads_or_tokens_needs_nothing(L):
    assert L.hc_gated_delta_workspace_bytes(0, 4096, 4, 4, 64, 64, 1) == 0
    assert L.hc_gated_delta_workspace_bytes(1, 0, 4, 4, 64, 64, 1) == 0
