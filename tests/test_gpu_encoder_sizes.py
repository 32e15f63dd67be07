"""Rows whose elements lie beyond 2^31, in every operator of the encoder."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import attention, close

pytestmark = pytest.mark.gpu


def test_attention_on_far_rows():
    """Rows 512 elements apart, the sequences behind element 2^31; everything before them is of no sequence."""
    n, step, lens = (1 << 22) + 5000, 512, [100, 300]
    far = torch.zeros(n, step, dtype=torch.bfloat16, device="cuda")
    begin = n - sum(lens)
    far[begin:, :96] = torch.randn(sum(lens), 96, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    q, k, v = (far[:, i:i + 32].view(n, 1, 32) for i in (0, 32, 64))
    offs = torch.tensor([begin, begin + 100, n], dtype=torch.int32, device="cuda")
    op = rece.SequenceAttention(n, 2, 1, 32)
    dout = torch.ones(n, 1, 32, dtype=torch.bfloat16, device="cuda")
    out, ws = op.forward(q, k, v, offs)
    assert begin * step > 1 << 31
    grads = op.backward(q, k, v, offs, out, ws, dout)
    cut = [t[begin:].cpu() for t in (q, k, v, dout)]
    want = attention(*cut[:3], [0, 100, 400], op.scale, dout=cut[3])
    for name, t in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        assert close(t[begin:], want[name]) <= 1.0, name
        assert (t[:begin] == 0).all(), name


def test_last_tokens_on_far_rows():
    rows, hk, d = 9_000_000, 4, 64
    kv = torch.zeros(rows, hk, d, dtype=torch.bfloat16, device="cuda")
    begin, length = rows - 700, 600
    kv[begin:] = torch.randn(700, hk, d, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    q = torch.randn(1, hk, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    for max_len in (600, 100_000):
        op = rece.LastAttention(1, rows, hk, d, max_len)
        out = op.forward(q.cuda(), kv, kv, one(begin), one(length))
        Q = torch.zeros(length, hk, d, dtype=torch.bfloat16)
        Q[-1] = q[0]
        part = kv[begin:begin + length].cpu()
        val, e = attention(Q, part, part, [0, length], op.scale)["out"]
        assert close(out[0], (val[-1], 2 * e[-1])) <= 1.0


def test_norm_and_rows_in_8_bits():
    n, d = 290_000, 8192
    x = torch.randn(n, d, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(d, device="cuda")
    op = rece.ResidualNorm(n, d)
    y, h, rstd = op.forward(x, None, w)
    far = x[-3:].float()
    want = far * (far.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w
    assert ((y[-3:].float() - want).abs() <= 2.0 ** -7 * want.abs()).all()
    dx, _ = op.backward(y, h, w, rstd)
    few = rece.ResidualNorm(3, d)
    dx3, _ = few.backward(y[-3:].contiguous(), x[-3:].contiguous(), w, rstd[-3:].contiguous())
    assert torch.equal(dx[-3:], dx3)
    x8, s = rece.quantize_rows(x)
    x3, s3 = rece.quantize_rows(x[-3:].contiguous())
    assert torch.equal(x8[-3:], x3) and torch.equal(s[-3:], s3)


@pytest.mark.parametrize("s,C,d", [(2200, 1_000_003, 32), (20, 110_000_001, 32), (40, 60_000_000, 64), (16400, 140_001, 272)])
def test_scores(s, C, d):
    x8 = torch.randint(-127, 128, (s, d), device="cuda", dtype=torch.int8)
    y8 = torch.randint(-127, 128, (C, d), device="cuda", dtype=torch.int8)
    sx, sy = torch.rand(s, device="cuda"), torch.rand(C, device="cuda")
    assert s * C > 1 << 31
    out = rece.Int8Scores(s, C, d).forward(x8, sx, y8, sy)
    for rows, cols in ((slice(s - 3, s), slice(C - 1000, C)), (slice(0, 3), slice(0, 1000)), (slice(s // 2, s // 2 + 2),
                                                                                            slice(C // 2, C // 2 + 999))):
        want = (x8[rows].double() @ y8[cols].double().T) * sx[rows].double()[:, None] * sy[cols].double()
        assert ((out[rows, cols].double() - want).abs() <= 2.0 ** -7 * want.abs()).all()
