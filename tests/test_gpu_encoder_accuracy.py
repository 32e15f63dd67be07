"""What the sequence encoder's operators add to the rounding of their results, as norms over whole results: bounds of single
values (encoder_reference) are sums of absolute values, which a rounding of p or ds to fewer bits passes."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import attention
from test_gpu_attention import last_reference, make

pytestmark = pytest.mark.gpu


def over_rounding(got, exact):
    """Norm of the error in units of that of the exact result's own rounding."""
    err = (got.double().cpu() - exact).norm()
    return float(err / (exact.to(got.dtype).double() - exact).norm())


# Errors are independent of the results' rounding, so their squares add up.  Operands of second products in two bf16 terms
# are off by 2^-17 relative at most, the results by 2^-9: 1.05 leaves the terms of a result 80 times its own size, and one
# term alone (2^-9 of p or ds, as much as the results' own) gives 1.3 and more.
MOST = 1.05


@pytest.mark.parametrize("lens,hq,hk,d,n_buckets", [
    ([300, 1, 77, 513], 4, 2, 32, 16), ([300, 1, 77, 513], 4, 2, 64, 16), ([260, 90], 4, 1, 128, 16), ([260, 90], 2, 2, 128, 0),
    ([20] * 60, 2, 2, 64, 16), ([300, 77], 2, 1, 40, 0),
])
def test_bf16_attention_is_off_by_its_results_rounding(lens, hq, hk, d, n_buckets):
    print(f"[gpu] accuracy lens={lens[:4]} hq={hq} hk={hk} d={d} buckets={n_buckets}", flush=True)
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make(lens, hq, hk, d, "bf16", n_buckets)
    o, b = offs.cuda(), None if bias is None else bias.cuda()
    out, ws = op.forward(Q, K, V, o, bias=b)
    grads = op.backward(Q, K, V, o, out, ws, dout.cuda(), bias=b)
    want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds or (), dout=dout)
    worst = {name: over_rounding(t, want[name][0]) for name, t in zip(("out", "dq", "dk", "dv"), (out, *grads))}
    print("  ", {name: round(x, 3) for name, x in worst.items()})
    if bias is not None:
        # float32: scores of d products off by sqrt(d) steps of up to 8, 4e-6 of p and ds (D from bf16 outputs: 2^-9)
        off = float((grads[3].double().cpu() - want["dbias"][0]).norm() / want["dbias"][0].norm())
        print(f"   dbias: {off:.2e}")
        assert off <= 1e-5
    assert max(worst.values()) <= MOST, worst


@pytest.mark.parametrize("lens,hq,hk,d,n_buckets", [([300, 1, 77, 513], 4, 2, 32, 16), ([300, 1, 77], 4, 2, 64, 16),
                                                    ([260, 90], 4, 1, 128, 0), ([20] * 60, 2, 2, 64, 16)])
def test_float32_attention(lens, hq, hk, d, n_buckets):
    """Scores of d products: sqrt(d) steps and a handful for scale, bias and log-sum-exp, each U / sqrt(3) of scores of some 3:
    (sqrt(128) + 8) U sqrt(3) = 2e-6 of p at most, and of sums of p."""
    print(f"[gpu] accuracy f32 lens={lens[:4]} hq={hq} hk={hk} d={d} buckets={n_buckets}", flush=True)
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make(lens, hq, hk, d, "f32", n_buckets)
    o, b = offs.cuda(), None if bias is None else bias.cuda()
    out, ws = op.forward(Q, K, V, o, bias=b)
    grads = op.backward(Q, K, V, o, out, ws, dout.cuda(), bias=b)
    want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds or (), dout=dout)
    for name, t in zip(("out", "dq", "dk", "dv", "dbias"), (out, *grads)):
        if t is not None:
            off = float((t.double().cpu() - want[name][0]).norm() / want[name][0].norm())
            print(f"   {name}: {off:.2e}")
            assert off <= 2e-6, name


@pytest.mark.parametrize("hq,hk,d,lens,max_len", [(4, 2, 32, [300, 1, 900, 64], 900), (8, 2, 64, [2000, 1500, 700], 2000),
                                                  (8, 2, 128, [1100, 31, 333], 400)])
def test_bf16_last_tokens_are_off_by_their_results_rounding(hq, hk, d, lens, max_len):
    g = torch.Generator().manual_seed(d)
    n_seq, rows = 8 * len(lens), 8 * sum(lens)
    q = torch.randn(n_seq, hq, d, generator=g).bfloat16()
    kv = torch.randn(rows, 2, hk, d, generator=g).bfloat16()
    length = torch.tensor(lens * 8, dtype=torch.int32)
    begin = (length.cumsum(0) - length).to(torch.int32)
    bias = torch.randn(16, hq, generator=g)
    op = rece.LastAttention(n_seq, rows, hq, d, max_len, kv_heads=hk, bounds=rece.log_buckets(16, 60))
    KV = kv.cuda()
    out = op.forward(q.cuda(), KV[:, 0], KV[:, 1], begin.cuda(), length.cuda(), bias=bias.cuda())
    ratio = over_rounding(out, last_reference(q, kv[:, 0], kv[:, 1], begin, length, op, bias)[0])
    print(f"[gpu] last accuracy {hq} {hk} {d}: {ratio:.3f}", flush=True)
    assert ratio <= MOST
