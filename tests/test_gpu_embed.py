"""Item embedding against the plain float64 form: rows times a scale, and the table's
gradient by sorted ids (written, accumulated, in float32 and bf16)."""
import numpy as np
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(n, C, d, dtype, ids_kind, seed):
    g = torch.Generator().manual_seed(seed)
    table = torch.randn(C, d, generator=g).to(DT[dtype])
    dout = torch.randn(n, d, generator=g).to(DT[dtype])
    if ids_kind == "uniform":
        ids = torch.randint(-2, C + 2, (n,), generator=g)       # some padding on either side
    elif ids_kind == "one":
        ids = torch.full((n,), C - 1)
    elif ids_kind == "none":
        ids = torch.full((n,), -1)
    elif ids_kind == "heavy":                                    # half the ids are one item
        ids = torch.where(torch.rand(n, generator=g) < 0.5, C // 2, torch.randint(0, C, (n,), generator=g))
    else:
        ids = torch.arange(n) % C
    return table, ids.to(torch.int32), dout


CASES = [
    (1, 1, 8, "f32", "one"), (1, 5, 32, "bf16", "uniform"), (33, 7, 64, "bf16", "uniform"),
    (256, 2000, 64, "f32", "uniform"), (1000, 3, 128, "bf16", "uniform"), (4097, 1237, 96, "bf16", "heavy"),
    (5000, 40, 256, "f32", "heavy"), (3000, 70001, 32, "bf16", "uniform"), (2048, 100, 64, "f32", "one"),
    (777, 50, 64, "bf16", "none"), (9000, 9000, 40, "f32", "range"), (300, 11, 1032, "bf16", "uniform"),
    (64, 9, 8192, "f32", "uniform"), (70000, 300, 32, "bf16", "heavy"), (100000, 1 << 20, 32, "bf16", "uniform"),
]


@pytest.mark.parametrize("n,C,d,dtype,kind", CASES)
def test_embed_forward_and_gradient(n, C, d, dtype, kind):
    table, ids, dout = _case(n, C, d, dtype, kind, seed=n + C)
    scale = float(np.float32(d ** 0.5))
    print(f"[gpu] embed n={n} C={C} d={d} {dtype} {kind}", flush=True)
    u = R.U[DT[dtype]]
    op = rece.ItemEmbedding(n, C, d, dtype=dtype, scale=scale)
    out = op.forward(table.cuda(), ids.cuda())
    want = R.embed(table, ids, scale)
    err = (out.cpu().double() - want).abs()
    assert bool((err <= (u + R.U32) * 1.01 * want.abs()).all())
    grad, bound = R.embed_grad(ids, dout, C, scale)
    got = op.backward(ids.cuda(), dout.cuda(), dtable=torch.full((C, d), float("nan"), device="cuda"))
    assert bool(((got.cpu().double() - grad).abs() <= bound).all())
    # accumulated onto a gradient that is there: one more float32 addition; other rows as they were
    base = torch.randn(C, d, generator=torch.Generator().manual_seed(5))
    acc = base.cuda()
    op.backward(ids.cuda(), dout.cuda(), dtable=acc, accumulate=True)
    err = (acc.cpu().double() - (base.double() + grad)).abs()
    assert bool((err <= bound + 2 * R.U32 * (base.double().abs() + grad.abs() + bound)).all())
    named = torch.zeros(C, dtype=torch.bool)
    named[ids[(ids >= 0) & (ids < C)].long()] = True
    assert torch.equal(acc.cpu()[~named], base[~named])
    # bf16 gradients: the float32 ones rounded
    opb = rece.ItemEmbedding(n, C, d, dtype=dtype, scale=scale, bf16_grads=True)
    gb = opb.backward(ids.cuda(), dout.cuda())
    assert torch.equal(gb, got.to(torch.bfloat16))
    # a second call gives the same bits
    assert torch.equal(op.backward(ids.cuda(), dout.cuda()), got)


def test_padding_rows_hold_anything():
    n, C, d = 200, 30, 64
    table, ids, dout = _case(n, C, d, "bf16", "uniform", seed=9)
    bad = (ids < 0) | (ids >= C)
    assert bool(bad.any())
    dout[bad] = float("nan")
    op = rece.ItemEmbedding(n, C, d, scale=float("inf"))
    out = op.forward(table.cuda(), ids.cuda())
    assert bool((out.cpu()[bad] == 0).all())
    op = rece.ItemEmbedding(n, C, d, scale=2.0)
    got = op.backward(ids.cuda(), dout.cuda())
    grad, bound = R.embed_grad(ids, torch.where(bad[:, None], 0.0, dout.float()), C, 2.0)
    assert bool(((got.cpu().double() - grad).abs() <= bound).all())


def test_no_rows_clears_the_gradient():
    op = rece.ItemEmbedding(0, 10, 32)
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    z = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    assert op.forward(torch.ones(10, 32, dtype=torch.bfloat16, device="cuda"), ids).shape == (0, 32)
    got = op.backward(ids, z, dtable=torch.ones(10, 32, device="cuda"))
    assert not bool(got.any())
    kept = op.backward(ids, z, dtable=torch.ones(10, 32, device="cuda"), accumulate=True)
    assert bool((kept == 1).all())


def test_autograd_and_differences():
    n, C, d = 50, 20, 32
    table, ids, _ = _case(n, C, d, "f32", "uniform", seed=3)
    w = torch.randn(n, d, generator=torch.Generator().manual_seed(4))
    op = rece.ItemEmbedding(n, C, d, dtype="f32", scale=3.0)
    t = table.cuda().requires_grad_(True)
    (rece.embed(t, ids.cuda(), op) * w.cuda()).sum().backward()
    # the function is linear in the table: a difference of any step is its slope
    f = lambda tab: float((R.embed(tab, ids, 3.0) * w.double()).sum())  # noqa: E731
    for j, c in ((0, 0), (7, 31), (C - 1, 5)):
        e = torch.zeros(C, d, dtype=torch.float64)
        e[j, c] = 0.5
        slope = f(table.double() + e) - f(table.double() - e)
        k = int((ids == j).sum())
        assert abs(float(t.grad[j, c]) - slope) <= (k + 2) * R.U32 * 3.0 * float(w.abs().sum()) + 1e-9


def test_capture_replay_and_streams():
    n, C, d = 3000, 500, 64
    table, ids, dout = (x.cuda() for x in _case(n, C, d, "bf16", "heavy", seed=11))
    op = rece.ItemEmbedding(n, C, d, scale=8.0)
    ref, refg = op.forward(table, ids), op.backward(ids, dout)
    out, g = torch.empty_like(ref), torch.empty_like(refg)
    ws = torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            op.forward(table, ids, out=out)
            op.backward(ids, dout, workspace=ws, dtable=g)
    for r in range(3):
        out.zero_()
        g.fill_(7.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(g, refg), r
        assert torch.equal(op.backward(ids, dout), refg)
