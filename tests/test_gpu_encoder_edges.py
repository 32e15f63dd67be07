"""Calls that the documentation of the sequence encoder's operators allows at their edges: masks that leave nothing,
NaN and infinities where they must not spread, rows of no sequence, offsets and lengths out of range, strides,
the most buckets, streams, graphs, two runs alike."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import HALF, attention, close, moved, norm
from test_gpu_attention import DT, check, last_reference, make

pytestmark = pytest.mark.gpu


def run(op, Q, K, V, offs, bias, dout):
    out, ws = op.forward(Q, K, V, offs, bias=bias)
    return (out, *op.backward(Q, K, V, offs, out, ws, dout, bias=bias))


NAMES = ("out", "dq", "dk", "dv", "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("-inf"), torch.finfo(torch.float32).min, -1e30])
@pytest.mark.parametrize("masked", [[0], [15], [0, 1, 2, 3], list(range(16))])
def test_masked_buckets(masked, value, dtype):
    """Buckets without weight: the nearest (a sequence's first row has nothing), the farthest, all."""
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make([1, 40, 200], 2, 1, 32, dtype, 16)
    bias[masked] = value
    got = run(op, Q, K, V, offs.cuda(), bias.cuda(), dout.cuda())
    want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds, dout=dout)
    for name, t in zip(NAMES, got):
        assert torch.isfinite(t).all(), name
        assert close(t, want[name]) <= 1.0, name
    if 0 in masked:
        assert (got[0][offs[:-1].long()[:3]] == 0).all()
    assert (got[4][masked] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [24, 64, 128])
def test_rows_of_no_sequence(d, dtype):
    """They become 0, and the NaN they hold reaches nothing."""
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make([33, 0, 90], 2, 2, d, dtype, 16, before=5, behind=70)
    for t in (Q, K, V, dg := dout.cuda()):
        t[:5] = float("nan")
        t[-70:] = float("inf")
    got = run(op, Q, K, V, offs.cuda(), bias.cuda(), dg)
    want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds, dout=dout)
    for name, t in zip(NAMES, got):
        assert torch.isfinite(t).all() and close(t, want[name]) <= 1.0, name
        if name != "dbias":
            assert (t[:5] == 0).all() and (t[-70:] == 0).all(), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[40, 50, 60], [20, 20, 20, 20], [130, 300, 200]])
def test_what_a_sequence_holds_stays_there(lens, dtype):
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make(lens, 2, 1, 64, dtype, 16)
    a, b = int(offs[1]), int(offs[2])
    for t in (Q, K, V, dg := dout.cuda()):
        t[a:b] = float("nan")
    got = run(op, Q, K, V, offs.cuda(), bias.cuda(), dg)
    want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds, dout=dout)
    for name, t in zip(NAMES[:4], got):
        val, e = want[name]
        rest = [i for i in range(t.shape[0]) if not a <= i < b]
        assert torch.isfinite(t[rest]).all() and close(t[rest], (val[rest], e[rest])) <= 1.0, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offsets", [[-5, 30, 400], [0, 100, 1 << 30], [10, 10, 10], [200, 200, 200]])
def test_offsets_out_of_range_are_clamped(offsets, dtype):
    op, (q, k, v), _, bias, bounds, dout, (Q, K, V) = make([100, 100], 2, 2, 32, dtype, 8)
    got = run(op, Q, K, V, torch.tensor(offsets, dtype=torch.int32, device="cuda"), bias.cuda(), dout.cuda())
    want = attention(q, k, v, offsets, op.scale, bias=bias, bounds=bounds, dout=dout)
    for name, t in zip(NAMES, got):
        assert close(t, want[name]) <= 1.0, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    """More sequences than one round of the search holds, most of them empty."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (1500,), generator=g).tolist() + [0] * 600 + [70, 0, 0, 1]
    check(lens, 1, 1, 32, dtype, n_buckets=8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d", [(2, 1, 32), (8, 1, 128)])
def test_the_most_buckets_and_distances(hq, hk, d, dtype):
    op, (q, k, v), offs, _, _, dout, (Q, K, V) = make([600, 4], hq, hk, d, dtype)
    for bounds in (list(range(1, 128)), [1, 2, 4096], list(range(30, 4000, 40)), [500], []):
        op = rece.SequenceAttention(604, 2, hq, d, kv_heads=hk, dtype=dtype, bounds=bounds)
        bias = torch.randn(len(bounds) + 1, hq, generator=torch.Generator().manual_seed(1))
        got = run(op, Q, K, V, offs.cuda(), bias.cuda(), dout.cuda())
        want = attention(q, k, v, offs.tolist(), op.scale, bias=bias, bounds=bounds, dout=dout)
        for name, t in zip(NAMES, got):
            assert close(t, want[name]) <= 1.0, (name, len(bounds))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_apart_and_gradients_in_one_piece(dtype):
    """Rows of separate tensors with room between them, gradients written into slices; what lies around stays."""
    lens, hq, hk, d = [65, 100], 4, 2, 40
    op, (q, k, v), offs, bias, bounds, dout, (Q, K, V) = make(lens, hq, hk, d, dtype, 8, fused=False)
    n = sum(lens)
    far = [torch.full((n, h * d + 24), 3.0, dtype=DT[dtype], device="cuda") for h in (hq, hk, hk)]
    views = [f[:, 8:8 + h * d].view(n, h, d) for f, h in zip(far, (hq, hk, hk))]
    for w, t in zip(views, (Q, K, V)):
        w.copy_(t)
    o, b, g = moved((offs, bias, dout))
    first = run(op, Q, K, V, o, b, g)
    out, ws = op.forward(*views, o, bias=b)
    grads = [torch.full_like(f, 5.0) for f in far]
    dst = [f[:, 8:8 + h * d].view(n, h, d) for f, h in zip(grads, (hq, hk, hk))]
    *_, dbias = op.backward(*views, o, out, ws, g, bias=b, dq=dst[0], dk=dst[1], dv=dst[2])
    for x, y in zip((out, *dst, dbias), first):
        assert torch.equal(x, y)
    for f, h in zip(grads, (hq, hk, hk)):
        assert (f[:, :8] == 5.0).all() and (f[:, 8 + h * d:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_runs_alike_on_two_streams(dtype):
    op, _, offs, bias, _, dout, (Q, K, V) = make([300, 20, 77], 4, 2, 64, dtype, 16)
    o, b, g = moved((offs, bias, dout))
    first = run(op, Q, K, V, o, b, g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, ws = op.forward(Q, K, V, o, bias=b, stream=s)
    other = (out, *op.backward(Q, K, V, o, out, ws, g, bias=b, stream=s))
    again = run(op, Q, K, V, o, b, g)
    torch.cuda.synchronize()
    for x, y, z in zip(first, other, again):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("d", [32, 128])
def test_attention_in_a_graph(d):
    """A captured forward and backward pass on new inputs, with eager work between the replays (d 128: more LDS than a
    launch gets without asking)."""
    op, _, offs, bias, _, dout, (Q, K, V) = make([150, 33, 200], 2, 1, d, "bf16", 16)
    o, b, g = moved((offs, bias, dout))
    run(op, Q, K, V, o, b, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run(op, Q, K, V, o, b, g)
    for seed in range(3):
        Q.copy_(torch.randn(Q.shape, generator=torch.Generator().manual_seed(seed)).to(Q.dtype))
        b.add_(0.1)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(kept, run(op, Q, K, V, o, b, g)):
            assert torch.equal(x, y)


def test_attention_on_shared_workspace_after_another_call():
    """A workspace given by the caller serves calls of the same operator one after the other."""
    op, _, offs, bias, _, dout, (Q, K, V) = make([64, 64], 2, 2, 32, "f32", 8)
    o, b, g = moved((offs, bias, dout))
    first = run(op, Q, K, V, o, b, g)
    ws = torch.full((op.workspace_bytes + 32,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out, same = op.forward(Q, K, V, o, bias=b, workspace=ws)
        assert same is ws
        for x, y in zip((out, *op.backward(Q, K, V, o, out, ws, g, bias=b)), first):
            assert torch.equal(x, y)


def test_no_tokens():
    for bounds in (None, [1, 2]):
        op = rece.SequenceAttention(0, 3, 2, 32, bounds=bounds)
        t = torch.empty(0, 2, 32, dtype=torch.bfloat16, device="cuda")
        bias = None if bounds is None else torch.randn(3, 2, device="cuda")
        offs = torch.zeros(4, dtype=torch.int32, device="cuda")
        out, ws = op.forward(t, t, t, offs, bias=bias)
        dq, dk, dv, dbias = op.backward(t, t, t, offs, out, ws, t, bias=bias)
        assert out.shape == t.shape and dv.shape == t.shape and (dbias is None or (dbias == 0).all())
    rn = rece.ResidualNorm(0, 64)
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    y, h, rstd = rn.forward(x, x, w)
    dx, dw = rn.backward(y, h, w, rstd)
    assert (dw == 0).all() and rn.forward_int8(x, x, w)[1].numel() == 0 and rece.quantize_rows(x)[0].shape == (0, 64)
    assert rece.Int8Scores(0, 5, 16).forward(torch.empty(0, 16, dtype=torch.int8, device="cuda"),
                                             torch.empty(0, device="cuda"),
                                             torch.zeros(5, 16, dtype=torch.int8, device="cuda"),
                                             torch.ones(5, device="cuda")).shape == (0, 5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_len", [1, 40, 3000])
def test_last_tokens_out_of_range_and_shared(max_len, dtype):
    """Beginnings and lengths beyond the cache are clamped, sequences share rows, others' rows hold NaN."""
    g = torch.Generator().manual_seed(1)
    rows, hq, hk, d = 700, 4, 2, 64
    q = torch.randn(7, hq, d, generator=g).to(DT[dtype])
    kv = torch.randn(rows, 2, hk, d, generator=g).to(DT[dtype])
    begin = torch.tensor([-3, 0, 10, 690, 800, 20, 30], dtype=torch.int32)
    length = torch.tensor([5, 40, -2, 100, 10, 1 << 30, 300], dtype=torch.int32)
    op = rece.LastAttention(7, rows, hq, d, max_len, kv_heads=hk, dtype=dtype, bounds=rece.log_buckets(8, 50))
    bias = torch.randn(8, hq, generator=g)
    args = (q, kv[:, 0], kv[:, 1], begin, length)
    Q, K, V, B, L, b = moved((*args, bias))
    got = op.forward(Q, K, V, B, L, bias=b)
    assert torch.isfinite(got).all() and close(got, last_reference(*args, op, bias)) <= 1.0
    assert (got[2] == 0).all() and (got[4] == 0).all()
    keep = got[1].clone()
    K[60:] = float("nan")
    V[60:] = float("inf")
    assert torch.equal(op.forward(Q, K, V, B, L, bias=b)[1], keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_last_tokens_with_masked_buckets(dtype):
    g = torch.Generator().manual_seed(2)
    q, kv = torch.randn(3, 2, 32, generator=g).to(DT[dtype]), torch.randn(400, 2, 2, 32, generator=g).to(DT[dtype])
    begin, length = torch.tensor([0, 1, 100], dtype=torch.int32), torch.tensor([1, 60, 300], dtype=torch.int32)
    for masked in ([0], [7], list(range(8))):
        op = rece.LastAttention(3, 400, 2, 32, 300, dtype=dtype, bounds=rece.log_buckets(8, 50))
        bias = torch.randn(8, 2, generator=g)
        bias[masked] = float("-inf")
        args = (q, kv[:, 0], kv[:, 1], begin, length)
        got = op.forward(*moved(args), bias=bias.cuda())
        assert torch.isfinite(got).all() and close(got, last_reference(*args, op, bias)) <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_extreme_rows(dtype):
    """Rows of zeros, of huge and tiny values, and ones that hold NaN or an infinity, which stay in their row."""
    d, big, small = 64, 1e30, 1e-30
    x = torch.randn(6, d, generator=torch.Generator().manual_seed(0))
    x[0], x[1], x[2] = 0.0, x[1] * big, x[2] * small
    x[3, 5], x[4, 7] = float("nan"), float("inf")
    x = x.to(DT[dtype])
    w = torch.linspace(0.5, 1.5, d)
    op = rece.ResidualNorm(6, d, eps=1e-6, dtype=dtype)
    X, W = x.cuda(), w.cuda()
    y, h, rstd = op.forward(X, None, W)
    assert h is X
    want = norm(x, None, w, 1e-6)["y"]
    fine = [0, 1, 2, 5]
    tol = (HALF[x.dtype] + 2.0 ** -21) * want[fine].abs() + 1e-38
    assert ((y.double().cpu()[fine] - want[fine]).abs() <= tol).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4, 7])
    y8, scale, _ = op.forward_int8(X, None, W)
    q8, s8 = rece.quantize_rows(X)
    for v8, s in ((y8, scale), (q8, s8)):
        assert s[0] == 0 and (v8[[0, 3, 4]] == 0).all() and torch.isnan(s[[3, 4]]).all() and torch.isfinite(s[fine]).all()
        assert (v8[[1, 2, 5]].abs().amax(1) == 127).all()


def test_norm_in_place():
    x, r = (torch.randn(50, 96, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(96, device="cuda")
    op = rece.ResidualNorm(50, 96)
    y, h, _ = op.forward(x, r, w)
    q, s, _ = op.forward_int8(x, r, w)
    r2, x2 = r.clone(), x.clone()
    y2, h2, _ = op.forward(x, r2, w, h=r2)
    q3, s3, h3 = op.forward_int8(x2, r, w, h=x2)
    assert h2 is r2 and h3 is x2 and torch.equal(h, h2) and torch.equal(h, h3)
    assert torch.equal(y, y2) and torch.equal(q, q3) and torch.equal(s, s3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_int8_ties_go_to_even(dtype):
    """127 h w / m next to and at halves, where float32 quotients go either way."""
    d = 256
    m = 254.0
    row = torch.cat([torch.arange(0, 127).float(), -torch.arange(0, 128).float(), torch.tensor([m])])
    x = torch.stack([row, row / 3.0, row * 7.0]).to(DT[dtype])
    x8, s = rece.quantize_rows(x.cuda())
    v = x.double()
    want = (127.0 * v / v.abs().amax(1, keepdim=True)).round().to(torch.int8)
    assert x.shape[1] == d and torch.equal(x8.cpu(), want)


def test_scores_and_norm_on_a_stream_and_in_a_graph():
    x = torch.randn(70, 64, device="cuda")
    w = torch.rand(64, device="cuda")
    y8, sy = rece.quantize_rows(torch.randn(3001, 64, device="cuda"))
    op, sc = rece.ResidualNorm(70, 64, dtype="f32"), rece.Int8Scores(70, 3001, 64, dtype="f32")

    def both(stream=None):
        x8, sx, _ = op.forward_int8(x, None, w, stream=stream)
        return sc.forward(x8, sx, y8, sy, stream=stream)

    first = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = both(s)
    torch.cuda.synchronize()
    assert torch.equal(other, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for _ in range(3):
        x.mul_(1.5).add_(0.1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, both())
