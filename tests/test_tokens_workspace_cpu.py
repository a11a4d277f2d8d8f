"""Workspace sizes of include/moe_tokens.h (CPU): no more than a call writes."""
import pytest

import expert_offload_lru_amd as moe


@pytest.mark.parametrize("T,inner,outer,n,r", [(512, 4096, 4096, 512, 64), (1, 2048, 2048, 1024, 64), (300, 768, 2048, 3, 8)])
def test_gradients_of_few_rows_join_no_pieces(T, inner, outer, n, r):
    """Offsets, order, counts, v and u, and the matrices laid out (4 bytes an element, whole runs of 64 columns and 16 ranks)."""
    def up(v, to):
        return (v + to - 1) // to * to

    layouts = n * 4 * (inner * up(r, 8) + up(r, 16) * (up(inner, 64) + up(outer, 64)))
    rows = 2 * 4 * T * up(r, 8) + 4 * (n + 1) + 4 * T + moe.gpu_lib().moe_tokens_workspace(T, 1, n)
    assert moe.gpu_lib().moe_adapters_workspace(T, inner, outer, n, r) <= layouts + rows + 16 * 256
