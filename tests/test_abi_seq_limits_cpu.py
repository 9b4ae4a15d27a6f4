"""The block operators' plans at the largest sizes that are accepted, through the workspaces they ask for (no GPU)."""
import pytest

import test_sequence_layers_amd as T
from seq_plans import SCAN_CASES, scan_segments

F32, BF16 = T.TTT_F32, T.TTT_BF16


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [1, 8, 64, 100, 4096, 16384])
@pytest.mark.parametrize("M", [(1 << 31) - 1 - k for k in (0, 1, 7, 15, 127, 128)])
def test_layernorm_backward_workspace_of_the_most_rows(dt, M, D):
    """Partial rows, two of D fp32 values each, of 512 workgroups (1024 threads: 256) or one for every 2048 turns, rounded
    up to 256 bytes; and no fewer than for a few rows."""
    need = T.load_library().ttt_backward_layernorm_workspace
    assert 0 < need(dt, M, 1, D) <= max(512, M // 2048 + 1) * 2 * D * 4 + 255
    assert need(dt, M, 1, D) >= need(dt, 1 << 14, 1, D) // 2


@pytest.mark.parametrize("dt,M,H,D,groups", [(F32, 32768, 4096, 1, 16), (BF16, 1000003, 128, 128, 64), (BF16, 1 << 26, 1, 8, 128),
                                             (F32, 300000, 1, 16384, 1), (F32, 32767, 65535, 8, 128)])
def test_layernorm_backward_walks_no_further_than_sums_allow(dt, M, H, D, groups):
    """At most 2048 turns: a partial row each time that a workgroup's groups (tokens of as many heads as there are, at most)
    have walked so far."""
    rows = T.load_library().ttt_backward_layernorm_workspace(dt, M, H, D) // (8 * H * D)
    assert rows * max(1, groups // H) * 2048 >= M


@pytest.mark.parametrize("B,N,C,S,G", [(4096, 32768, 1, 8, 1), (4096, 32767, 1, 16, 1), (24, 16384, 4096, 32, 1), (1, 1 << 22, 64, 16, 1),
                                       (64, 4096, 768, 64, 1), (1, 1 << 17, 1 << 20, 8, 1),
                                       (60000, 4096, 16, 8, 16), (65535, 3000, 64, 64, 1)])
def test_scan_segments_are_no_longer_than_sums_allow(B, N, C, S, G):
    """2048 tokens, in the forward pass where there is more than one."""
    nseg, tokens = scan_segments(B, N, C, S, G, backward=True)
    assert tokens <= 2048
    nseg, tokens = scan_segments(B, N, C, S, G)
    assert nseg == 1 or tokens <= 2048


@pytest.mark.parametrize("case", SCAN_CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_scan_cases_take_the_plans_that_they_are_for(case):
    B, N, C, S, G, dtype, _, forward, backward = case
    dt = F32 if dtype == "fp32" else BF16
    nseg, tokens = scan_segments(B, N, C, S, G, dtype=dt)
    assert tokens >= forward and (nseg == 1) == (forward == N)
    nseg, tokens = scan_segments(B, N, C, S, G, backward=True, dtype=dt)
    assert tokens >= backward and (nseg == 1) == (backward == N)
