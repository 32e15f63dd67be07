"""The last token's attention over the longest cache there is: 2^31 - 1 rows of one sequence."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece

pytestmark = pytest.mark.gpu


def test_a_sequence_of_all_rows_there_can_be():
    """Keys of 0 but the last row's; the first query has no preference (the mean of the values), the second one sees the last
    row alone."""
    rows, d = (1 << 31) - 1, 8
    k = torch.zeros(rows, 1, d, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(rows, 1, d, dtype=torch.bfloat16, device="cuda")
    k[-1], v[-1] = 16.0, 7.0
    q = torch.zeros(2, 1, d, dtype=torch.bfloat16, device="cuda")
    q[1] = 4.0
    begin, length = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 0], [rows, rows]))
    print("[gpu] last tokens of 2^31 - 1 rows", flush=True)
    out = rece.LastAttention(2, rows, 1, d, rows).forward(q, k, v, begin, length)
    # scores 0 and 512 / sqrt(8) = 181: the others' weight is 2^31 e^-181
    assert (out[0] == 1.0).all() and (out[1] == 7.0).all()
