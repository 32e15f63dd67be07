"""What lengths the last token's attention plans for (no GPU needed)."""
import pytest

import catalogue_cross_entropy_amd as rece


@pytest.mark.parametrize("max_len", [(1 << 31) - 1, 1 << 40, (1 << 63) - 1])
def test_any_length_can_be_planned_for(max_len):
    """As many parts as for any long sequence."""
    op = rece.LastAttention(1, 1 << 20, 4, 64, max_len, kv_heads=2)
    assert op.workspace_bytes == rece.LastAttention(1, 1 << 20, 4, 64, 1 << 20, kv_heads=2).workspace_bytes > 0
