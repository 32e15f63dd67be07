"""The last token's attention at its limits: a sequence of 2^31 - 1 rows, and the most sequences and heads."""
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


def test_as_many_sequences_and_heads_as_there_can_be():
    """2^17 - 1 users of 32 query heads on one key head, one or two rows each."""
    n_seq, heads, d = (1 << 22) // 32 - 1, 32, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    kv = torch.randn(n_seq + 1, 2, 1, d, generator=g, device="cuda").bfloat16()
    q = torch.randn(n_seq, heads, d, generator=g, device="cuda").bfloat16()
    begin = torch.arange(n_seq, dtype=torch.int32, device="cuda")
    length = 1 + begin % 2
    print("[gpu] last tokens of the most sequences and heads", flush=True)
    out = rece.LastAttention(n_seq, n_seq + 1, heads, d, 2, kv_heads=1).forward(q, kv[:, 0], kv[:, 1], begin, length)
    k, v = (torch.stack([kv[:-1, i, 0], kv[1:, i, 0]], 1).double() for i in (0, 1))
    s = torch.matmul(q.double(), k.transpose(1, 2).contiguous()) * d ** -0.5
    s[length == 1, :, 1] = -torch.inf
    p = torch.softmax(s, 2)
    want = torch.matmul(p, v)
    # the result's rounding; p to 2^-16 and float32 steps of scores of up to some 30 beside terms of either sign
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -14 * torch.matmul(p, v.abs())
    assert ((out.double() - want).abs() <= tol).all()
