"""Attention over packed sequences and of last tokens against the float64 form."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import attention, close

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LENS = {
    "one": [1],
    "short": [1, 2, 0, 3, 7, 1, 31, 32, 33],
    "tiles": [127, 128, 129, 0, 0, 65, 64, 63],
    "long": [700, 5, 257],
}


def make(lens, hq, hk, d, dtype, n_buckets=0, seed=0, fused=True, before=0, behind=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + before + behind
    dt = DT[dtype]
    qkv = (spread * torch.randn(n, (hq + 2 * hk) * d, generator=g)).to(dt)
    offs = torch.tensor([before] + [before + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    bias = bounds = None
    if n_buckets:
        bounds = rece.log_buckets(n_buckets, 4 * n_buckets)
        bias = torch.randn(n_buckets, hq, generator=g)
    dout = torch.randn(n, hq, d, generator=g).to(dt)
    op = rece.SequenceAttention(n, len(lens), hq, d, kv_heads=hk, dtype=dtype, bounds=bounds)
    split = lambda t: (t[:, :hq * d].view(n, hq, d), t[:, hq * d:(hq + hk) * d].view(n, hk, d),  # noqa: E731
                       t[:, (hq + hk) * d:].view(n, hk, d))
    return op, split(qkv), offs, bias, bounds, dout, split(qkv.cuda()) if fused else tuple(t.contiguous().cuda() for t in split(qkv))


def check(lens, hq, hk, d, dtype, n_buckets=0, train=True, **kw):
    print(f"[gpu] attention lens={lens} hq={hq} hk={hk} d={d} {dtype} buckets={n_buckets} {kw}", flush=True)
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make(lens, hq, hk, d, dtype, n_buckets, **kw)
    o, b = offs.cuda(), None if bias is None else bias.cuda()
    out, ws = op.forward(Q, K, V, o, bias=b, need_grad=train)
    got = {"out": out}
    if train:
        got["dq"], got["dk"], got["dv"], got["dbias"] = op.backward(Q, K, V, o, out, ws, dout.cuda(), bias=b)
    torch.cuda.synchronize()
    want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds or (), dout=dout if train else None)
    for name in want:
        assert torch.isfinite(got[name]).all(), name
        worst = close(got[name], want[name])
        print(f"  {name}: {worst:.3f} of its bound")
        assert worst <= 1.0, name
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens", list(LENS))
def test_lengths(lens, d, dtype):
    check(LENS[lens], 2, 2, d, dtype, n_buckets=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (6, 2), (8, 8)])
def test_heads(hq, hk, dtype):
    check([50, 1, 200, 96], hq, hk, 32, dtype, n_buckets=8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 24, 40, 72, 104, 120])
def test_odd_head_widths(d, dtype):
    check([70, 3, 130], 2, 1, d, dtype, n_buckets=16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_without_bias(d, dtype):
    check([150, 33, 1, 300], 4, 2, d, dtype)
    check([150, 33, 1, 300], 4, 2, d, dtype, train=False)


def last_reference(q, k, v, begin, length, op, bias):
    """(value, bound) by the packed form: each sequence's rows with its query behind them."""
    val, err = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    rows = k.shape[0]
    for u in range(q.shape[0]):
        b = min(max(int(begin[u]), 0), rows)
        n = min(max(int(length[u]), 0), rows - b)
        if n == 0:
            continue
        Q = torch.zeros(n, *q.shape[1:], dtype=q.dtype)
        Q[-1] = q[u]
        o, e = attention(Q, k[b:b + n], v[b:b + n], [0, n], op.scale, bias=bias, bounds=op.bounds or ())["out"]
        val[u], err[u] = o[-1], 2 * e[-1]    # the reference of a part and that of all parts: scores are rounded twice
    return val, err


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d,lens,max_len,n_buckets", [
    (2, 2, 32, [1, 0, 31, 32, 33, 200], 200, 16), (8, 2, 64, [5, 700, 129], 700, 32), (4, 4, 128, [64, 1000], 1000, 0),
    (32, 1, 40, [300, 7], 300, 8), (1, 1, 8, [2, 5000], 5000, 64), (6, 3, 104, [900], 10, 16), (2, 1, 64, [9000], 9000, 0),
])
def test_last_tokens(hq, hk, d, lens, max_len, n_buckets, dtype):
    print(f"[gpu] last hq={hq} hk={hk} d={d} lens={lens} max_len={max_len} buckets={n_buckets} {dtype}", flush=True)
    g = torch.Generator().manual_seed(d + hq)
    dt, n_seq, rows = DT[dtype], len(lens), sum(lens) + 3 * len(lens)
    q = torch.randn(n_seq, hq, d, generator=g).to(dt)
    kv = torch.randn(rows, 2, hk, d, generator=g).to(dt)
    length = torch.tensor(lens, dtype=torch.int32)
    begin = torch.cumsum(length + 3, 0).to(torch.int32) - length - 3     # slots with room behind each
    bounds = rece.log_buckets(n_buckets, 3 * n_buckets) if n_buckets else None
    bias = torch.randn(n_buckets, hq, generator=g) if n_buckets else None
    op = rece.LastAttention(n_seq, rows, hq, d, max_len, kv_heads=hk, dtype=dtype, bounds=bounds)
    KV = kv.cuda()
    out = op.forward(q.cuda(), KV[:, 0], KV[:, 1], begin.cuda(), length.cuda(), bias=None if bias is None else bias.cuda())
    assert torch.isfinite(out).all()
    worst = close(out, last_reference(q, kv[:, 0], kv[:, 1], begin, length, op, bias))
    print(f"  out: {worst:.3f} of its bound")
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,hq,hk,d", [
    ([20] * 40, 2, 2, 64),             # a wave for a sequence
    ([64] * 3 + [70], 2, 2, 32),       # four waves; keys: one
    ([160], 1, 1, 64),                 # keys: two waves
    ([300, 200], 4, 1, 128),           # keys: four waves
    ([300, 200], 4, 1, 64),
])
def test_every_split_of_the_work(lens, hq, hk, d, dtype):
    check(lens, hq, hk, d, dtype, n_buckets=16)
    check(lens, hq, hk, d, dtype)
