"""Log-probabilities over the catalogue, entropies and their gradients against the plain
float64 form (tolerances: ops_reference.logprob)."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _case(s, C, d, dtype, seed, pad=0.0, peak=0.0):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(s, d, generator=g) * 1.5 * d ** -0.25
    Y = torch.randn(C, d, generator=g) * d ** -0.25
    ids = torch.randint(0, C, (s,), generator=g)
    X = X + peak * torch.rand(s, 1, generator=g) * Y[ids]
    bad = torch.rand(s, generator=g) < pad
    ids = torch.where(bad, torch.where(torch.rand(s, generator=g) < 0.5, -1, C), ids).to(torch.int32)
    X, Y = X.to(DT[dtype]), Y.to(DT[dtype])
    X[bad, 0] = float("nan")
    X[bad, 1] = float("inf")
    dlogp = torch.randn(s, generator=g) / s
    dent = torch.randn(s, generator=g) / s * 0.1
    return X, Y, ids, dlogp, dent, bad


def _run(X, Y, ids, dlogp, dent, T, entropy, bf16_grads):
    s, d = X.shape
    op = rece.LogProb(s, Y.shape[0], d, dtype="bf16" if X.dtype == torch.bfloat16 else "f32", temperature=T,
                      entropy=entropy, bf16_grads=bf16_grads)
    X, Y, ids = X.cuda(), Y.cuda(), ids.cuda()
    logp, ent, ws = op.forward(X, Y, ids)
    dX, dY = op.backward(X, Y, ids, ws, dlogp.cuda(), None if dent is None else dent.cuda())
    plain, ent2, _ = op.forward(X, Y, ids, need_grad=False)
    torch.cuda.synchronize()
    assert torch.equal(plain, logp) and (ent is None or torch.equal(ent, ent2))
    return logp.cpu(), None if ent is None else ent.cpu(), dX.cpu(), dY.cpu()


CASES = [
    # s, C, d, dtype, T, entropy, pad, peak
    (1, 1, 32, "f32", 1.0, True, 0.0, 0.0),
    (1, 2, 64, "bf16", 1.0, True, 0.0, 0.0),
    (5, 33, 64, "bf16", 0.7, True, 0.0, 1.0),
    (3, 5003, 128, "bf16", 1.3, True, 0.3, 2.0),
    (64, 64, 32, "bf16", 1.0, False, 0.0, 0.0),
    (257, 1000, 64, "bf16", 1.0, False, 0.2, 3.0),
    (257, 1000, 64, "f32", 1.0, True, 0.2, 3.0),
    (130, 257, 256, "bf16", 0.5, True, 0.1, 1.0),
    (130, 257, 256, "f32", 0.5, False, 0.1, 1.0),
    (700, 63, 128, "bf16", 1.0, False, 0.5, 1.0),
    (700, 65, 128, "f32", 2.0, True, 0.5, 1.0),
    (1030, 2049, 64, "bf16", 1.0, True, 0.25, 2.0),
    (2000, 31, 32, "f32", 1.0, False, 0.0, 1.0),
    (40, 20000, 64, "bf16", 1.0, False, 0.0, 2.0),
    (40, 20000, 256, "bf16", 1.0, True, 0.0, 2.0),
    (520, 1500, 128, "f32", 1.0, False, 0.1, 2.0),
]


@pytest.mark.parametrize("bf16_grads", [False, True])
@pytest.mark.parametrize("s,C,d,dtype,T,entropy,pad,peak", CASES)
def test_logprob_against_plain(s, C, d, dtype, T, entropy, pad, peak, bf16_grads):
    X, Y, ids, dlogp, dent, bad = _case(s, C, d, dtype, seed=s * 7 + C, pad=pad, peak=peak)
    if not entropy:
        dent = None
    print(f"[gpu] logprob s={s} C={C} d={d} {dtype} T={T} entropy={entropy} bf16_grads={bf16_grads}", flush=True)
    logp, ent, dX, dY = _run(X, Y, ids, dlogp, dent, T, entropy, bf16_grads)
    w = R.logprob(X, Y, ids, T, dlogp, dent)
    assert bool(((logp.double() - w["logp"]).abs() <= w["e_logp"]).all())
    assert bool((logp[bad] == 0).all()) and bool((dX[bad] == 0).all())
    if entropy:
        assert bool(((ent.double() - w["entropy"]).abs() <= w["e_entropy"]).all())
    u = R.U[torch.bfloat16] if bf16_grads else R.U32
    for name, got in (("dX", dX), ("dY", dY)):
        bound = w["p_" + name] + (w["b_" + name] if bf16_grads else 0.0)
        bound = bound + u * (w[name].abs() + bound) + 1e-30
        bad_at = (got.double() - w[name]).abs() > bound
        assert not bool(bad_at.any()), (name, float(((got.double() - w[name]).abs() / bound).max()))


def test_every_position_is_padding():
    X, Y, ids, dlogp, dent, _ = _case(300, 500, 64, "bf16", seed=1)
    ids[:] = -1
    X[:] = float("nan")
    logp, ent, dX, dY = _run(X, Y, ids, dlogp, dent, 1.0, True, False)
    assert not bool(logp.any()) and not bool(ent.any()) and not bool(dX.any()) and not bool(dY.any())


def test_logits_far_apart():
    """Logits from -3000 to 3000: the reference of the running sum moves many times, all but a few
    probabilities underflow, and rising and falling orders of items agree with the plain form."""
    s, C, d = 8, 3000, 32
    X = torch.zeros(s, d)
    Y = torch.zeros(C, d)
    X[:, 0] = torch.tensor([1.0, -1.0, 2.0, 0.5, 0.0, 1.5, -0.25, 1.0])
    Y[:, 0] = torch.linspace(-1500, 1500, C).round()
    ids = torch.tensor([C - 1, 0, 5, 17, 3, C - 2, 1, 0], dtype=torch.int32)
    dl, de = torch.ones(s) / s, torch.ones(s) / s * 0.01
    for Yo in (Y, Y.flip(0).contiguous()):
        logp, ent, dX, dY = _run(X, Yo, ids, dl, de, 1.0, True, False)
        w = R.logprob(X, Yo, ids, 1.0, dl, de)
        assert bool(((logp.double() - w["logp"]).abs() <= w["e_logp"]).all())
        assert bool(((ent.double() - w["entropy"]).abs() <= w["e_entropy"]).all())
        assert bool(torch.isfinite(dX).all()) and bool(torch.isfinite(dY).all())
        b = w["p_dX"] + R.U32 * w["dX"].abs() + 1e-30
        assert bool(((dX.double() - w["dX"]).abs() <= b).all())


def test_nan_rows_stay_in_their_rows():
    """A NaN in a position that counts reaches that position's results alone (and dY)."""
    X, Y, ids, dlogp, dent, _ = _case(70, 400, 64, "bf16", seed=2)
    X[13, 5] = float("nan")
    op = rece.LogProb(70, 400, 64)
    logp, _, ws = op.forward(X.cuda(), Y.cuda(), ids.cuda())
    dX, _ = op.backward(X.cuda(), Y.cuda(), ids.cuda(), ws, dlogp.cuda())
    fine = torch.arange(70) != 13
    assert bool(torch.isnan(logp[13])) and bool(torch.isfinite(logp.cpu()[fine]).all())
    assert bool(torch.isfinite(dX.cpu()[fine]).all())


def test_gradient_against_differences():
    s, C, d, T = 6, 50, 32, 0.8
    X, Y, ids, dlogp, dent, _ = _case(s, C, d, "f32", seed=5)
    _, _, dX, dY = _run(X, Y, ids, dlogp, dent, T, True, False)

    def value(Xd, Yd):
        w = R.logprob(Xd, Yd, ids, T)
        return float((w["logp"] * dlogp.double()).sum() + (w["entropy"] * dent.double()).sum())

    # central differences of the float64 form: step e leaves e^2 / 6 of a third derivative that is
    # of the size of the value's scale here, and 2^-52 / e of rounding
    e = 1e-5
    for t, grad, which in ((X, dX, 0), (Y, dY, 1)):
        for at in ((0, 0), (s - 1, 7), (2, d - 1)):
            step = torch.zeros_like(t, dtype=torch.float64)
            step[at] = e
            args = lambda sg: (X.double() + (sg * step if which == 0 else 0), Y.double() + (sg * step if which == 1 else 0))  # noqa: E731
            slope = (value(*args(1)) - value(*args(-1))) / (2 * e)
            assert abs(float(grad[at]) - slope) <= 1e-6


def test_full_ce_agrees():
    """The same loss by the two independent sweeps: mean of -logp and its gradients."""
    s, C, d = 512, 3000, 64
    X, Y, ids, _, _, _ = _case(s, C, d, "bf16", seed=8, peak=1.0)
    X, Y, ids = X.cuda(), Y.cuda(), ids.cuda()
    f = rece.FullCE(s, C, d)
    _, lpp, ws = f.forward(X, Y, ids)
    dX0, dY0 = f.backward(X, Y, ids, ws)
    op = rece.LogProb(s, C, d)
    logp, _, ws = op.forward(X, Y, ids)
    dX1, dY1 = op.backward(X, Y, ids, ws, torch.full((s,), -1.0 / s, device="cuda"))
    w = R.logprob(X.cpu(), Y.cpu(), ids.cpu(), 1.0, torch.full((s,), -1.0 / s))
    assert bool(((logp + lpp).abs().cpu() <= 2 * w["e_logp"]).all())
    # FullCE splits its weights into two bf16 terms (2^-16)
    for a, b, n in ((dX0, dX1, "dX"), (dY0, dY1, "dY")):
        assert bool(((a - b).abs().cpu().double() <= 2 * w["p_" + n] + 2.0 ** -7 * w["b_" + n] + 2.0 ** -15 * w[n].abs()).all())


def test_autograd_streams_capture():
    s, C, d = 300, 1200, 64
    X, Y, ids, dlogp, dent, _ = (t.cuda() for t in _case(s, C, d, "bf16", seed=12, pad=0.2, peak=1.0))
    op = rece.LogProb(s, C, d, temperature=0.9, entropy=True, bf16_grads=True)
    logp, ent, ws = op.forward(X, Y, ids)
    dX, dY = op.backward(X, Y, ids, ws, dlogp, dent)
    Xg, Yg = X.clone().requires_grad_(True), Y.clone().requires_grad_(True)
    a, b = rece.log_probs(Xg, Yg, ids, op)
    assert torch.equal(a, logp) and torch.equal(b, ent)
    ((a * dlogp).sum() + (b * dent).sum()).backward()
    assert torch.equal(Xg.grad, dX) and torch.equal(Yg.grad, dY)
    with torch.no_grad():
        a, b = rece.log_probs(Xg, Yg, ids, op)
        assert torch.equal(a, logp)
    # on another stream, and captured: replays after other work give the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")
    gX, gY = torch.empty_like(dX), torch.empty_like(dY)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            l2, e2, _ = op.forward(X, Y, ids, workspace=ws)
            op.backward(X, Y, ids, ws, dlogp, dent, dX=gX, dY=gY)
    for r in range(3):
        for t in (l2, e2, gX, gY):
            t.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(l2, logp) and torch.equal(e2, ent) and torch.equal(gX, dX) and torch.equal(gY, dY), r
        l3, _, w3 = op.forward(X, Y, ids)
        assert torch.equal(op.backward(X, Y, ids, w3, dlogp, dent)[1], dY)
