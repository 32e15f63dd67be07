"""What lengths and numbers of sequences the last token's attention takes (no GPU needed)."""
import pytest

import catalogue_cross_entropy_amd as rece


@pytest.mark.parametrize("max_len", [(1 << 31) - 1, 1 << 40, (1 << 63) - 1])
def test_any_length_can_be_planned_for(max_len):
    """As many parts as for any long sequence."""
    op = rece.LastAttention(1, 1 << 20, 4, 64, max_len, kv_heads=2)
    assert op.workspace_bytes == rece.LastAttention(1, 1 << 20, 4, 64, 1 << 20, kv_heads=2).workspace_bytes > 0


def test_as_many_sequences_and_heads_as_documented():
    most = (1 << 22) // 32
    assert rece.LastAttention(most - 1, 100, 32, 8, 50, kv_heads=1).workspace_bytes == 0
    assert rece.LastAttention(65536, 100, 32, 64, 50).workspace_bytes == 0
    for n_seq, heads, kv in ((most, 32, 1), (4, 1032, 1032)):
        with pytest.raises(rece.ReceError):
            rece.LastAttention(n_seq, 100, heads, 8, 50, kv_heads=kv)
