"""Workspaces of the token mixers against the most that the headers of the plans promise (CPU only)."""

import pytest

import chunked_gated_delta_amd as kda


@pytest.mark.parametrize("K,V", [(128, 128), (64, 128), (64, 64)])
@pytest.mark.parametrize("T", [1, 384, 385, 4096, 1 << 24])
@pytest.mark.parametrize("H", [1, 7, 96, 200, 2000])
def test_states_of_at_most_1024_pieces(T, H, K, V):
    """Cutting leads to 1024 workgroups at most, each with a state, and to none where a call is short."""
    most = min(1024, T // 128 * H if T > 384 else 0) * K * V * 4
    assert kda.kda_la_workspace_size(T, H, K, V) <= most
    for N in (1, 4, 1000):
        assert kda.kda_la_bwd_workspace_size(T, H, K, V, N) <= 4 * most + 4 * (2 * N * H + 1024) + 255
