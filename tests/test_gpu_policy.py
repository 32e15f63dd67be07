"""Policy and preference losses against their plain float64 forms, and a run of all the
operators together as a preference or policy update uses them."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _offsets(g, n_seq, n, lead=0, trail=0):
    cut = torch.sort(torch.randint(lead, n - trail + 1, (n_seq + 1,), generator=g)).values
    cut[0], cut[-1] = lead, n - trail
    return cut.to(torch.int32)


def _tokens(g, n, dtype):
    lp = -8.0 * torch.rand(n, generator=g)
    return lp.to(DT[dtype]), (lp + 0.2 * torch.randn(n, generator=g)).to(DT[dtype]), \
        (lp + 0.5 * torch.randn(n, generator=g)).to(DT[dtype])


POLICY = [
    # n, n_seq, dtype, kl, ent, token_adv, reduction, masked, lead, trail
    (1, 1, "f32", 0.1, 0.01, False, "token", False, 0, 0),
    (40, 7, "f32", 0.1, 0.01, False, "sequence", True, 3, 5),
    (40, 60, "bf16", 0.0, 0.0, True, "sequence", True, 0, 0),
    (8192, 2048, "f32", 0.05, 0.0, False, "sequence", True, 0, 17),
    (8193, 5, "f32", 0.05, 0.02, False, "token", True, 1, 1),
    (5000, 3000, "f32", 0.05, 0.02, False, "sequence", False, 9, 0),
    (30001, 900, "bf16", 0.05, 0.02, True, "token", False, 7, 100),
    (30001, 900, "bf16", 0.05, 0.02, False, "sequence", True, 7, 100),
    (70000, 3, "f32", 0.0, 0.02, False, "sequence", True, 0, 0),
    (70000, 9000, "f32", 0.2, 0.0, False, "token", True, 0, 4097),
]


@pytest.mark.parametrize("n,n_seq,dtype,kl,ent,token,reduction,masked,lead,trail", POLICY)
def test_policy_against_plain(n, n_seq, dtype, kl, ent, token, reduction, masked, lead, trail):
    g = torch.Generator().manual_seed(n + n_seq)
    lp, old, ref = _tokens(g, n, dtype)
    H = (5.0 * torch.rand(n, generator=g)).to(DT[dtype]) if ent else None
    offs = _offsets(g, n_seq, n, lead, trail)
    adv = torch.randn(n if token else n_seq, generator=g)
    mask = (torch.rand(n, generator=g) < 0.7).to(torch.uint8) if masked else None
    if masked:   # what does not count may be anything
        off = mask == 0
        lp, old, ref = (t.clone() for t in (lp, old, ref))
        lp[off], old[off], ref[off] = float("nan"), float("-inf"), float("inf")
    cfg = dict(low=0.2, high=0.28, kl=kl, ent=ent, token=token, reduction=reduction)
    if not kl:
        ref = None
    print(f"[gpu] policy n={n} n_seq={n_seq} {dtype} {reduction} kl={kl} ent={ent} masked={masked}", flush=True)
    op = rece.PolicyLoss(n, n_seq, clip_low=0.2, clip_high=0.28, kl_coef=kl, entropy_coef=ent, reduction=reduction,
                         token_advantage=token, dtype=dtype)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    dloss = torch.full((1,), 2.0, device="cuda")
    args = (cu(lp), cu(old), cu(adv), cu(offs))
    kw = dict(ref_logp=cu(ref), entropy=cu(H), mask=cu(mask))
    loss, stats, dlp, dH = op.forward(*args, dloss=dloss, **kw)
    wl, ws, wg, wh = R.policy(lp, old, adv, offs, cfg, ref, H, mask)
    # one token's terms: a difference, two exponentials (2 U32 each, and the difference's rounding times
    # its size, at most 8 here), a handful of products; relative to |A| r + kl_coef (e^u + |u| + 1) + ent H.
    # The sums are in float64.
    seq = R.seq_of_tokens(offs, n)
    on = (seq >= 0) & ((mask != 0) if mask is not None else torch.ones(n, dtype=torch.bool))
    z = lambda t: torch.where(on, t.double(), 0.0)  # noqa: E731
    A = (adv if token else adv[seq.clamp(min=0)]).double()
    r = (z(lp) - z(old)).exp()
    eu = (z(ref) - z(lp)).exp() if kl else torch.zeros(n, dtype=torch.float64)
    size = A.abs() * r.clamp(min=1.0) * 1.3 + kl * (eu + 12.0) + (ent * z(H) if ent else 0.0)
    rel = 40 * R.U32
    count = torch.zeros(n_seq, dtype=torch.float64).index_add_(0, seq[on], torch.ones(int(on.sum()), dtype=torch.float64))
    if reduction == "token":
        w = torch.full((n,), 1.0 / max(int(on.sum()), 1), dtype=torch.float64)
    else:
        w = (1.0 / (count.clamp(min=1) * max(int((count > 0).sum()), 1)))[seq.clamp(min=0)]
    e = torch.where(on, rel * w * size, 0.0)
    assert abs(float(loss) - wl) <= float(e.sum()) + 2 * R.U32 * abs(wl)
    k = max(int(on.sum()), 1)
    scale = [float((A.abs() * r * 1.3)[on].sum()) / k, float((eu + 12.0)[on].sum()) / k, 10.0, 1.0, float(r[on].sum()) / k, 0.0]
    got = stats.cpu().tolist()
    for a, b, c in zip(got, ws, scale):
        assert abs(a - b) <= rel * c + 2 * R.U32 * abs(b), (got, ws)
    u = R.U[DT[dtype]]
    assert bool(((dlp.cpu().double() - 2 * wg).abs() <= 2 * (e + u * (wg.abs() + e))).all())
    assert bool((dlp.cpu()[~on] == 0).all())
    if ent:
        assert bool(((dH.cpu().double() - 2 * wh).abs() <= 2 * (8 * R.U32 + u) * wh.abs()).all())
        assert bool((dH.cpu()[~on] == 0).all())
    again = op.forward(*args, dloss=dloss, **kw)
    assert torch.equal(again[0], loss) and torch.equal(again[1], stats) and torch.equal(again[2], dlp)
    none = op.forward(*args, grads=False, **kw)
    assert none[2] is None and torch.equal(none[0], loss)


@pytest.mark.parametrize("n,n_seq", [(300, 9), (20000, 40)])
def test_policy_nothing_counts(n, n_seq):
    g = torch.Generator().manual_seed(1)
    lp, old, ref = _tokens(g, n, "f32")
    offs = _offsets(g, n_seq, n).cuda()
    for reduction in ("token", "sequence"):
        op = rece.PolicyLoss(n, n_seq, kl_coef=0.1, reduction=reduction)
        loss, stats, dlp, _ = op.forward(lp.cuda(), old.cuda(), torch.ones(n_seq, device="cuda"), offs, ref_logp=ref.cuda(),
                                         mask=torch.zeros(n, dtype=torch.uint8, device="cuda"))
        assert float(loss) == 0.0 and not bool(stats.any()) and not bool(dlp.any())


@pytest.mark.parametrize("n,n_seq", [(500, 8), (12000, 8)])
def test_policy_offsets_outside_are_clamped(n, n_seq):
    """Offsets below 0 and beyond n: the same as the clamped ones, and nothing outside is touched."""
    g = torch.Generator().manual_seed(2)
    lp, old, _ = _tokens(g, n, "f32")
    offs = _offsets(g, n_seq, n)
    wild = offs.clone()
    wild[0], wild[1], wild[-1], wild[-2] = -50, -3, n + 1000, n + 7
    adv = torch.randn(n_seq, generator=g).cuda()
    op = rece.PolicyLoss(n, n_seq, reduction="sequence")
    a = op.forward(lp.cuda(), old.cuda(), adv, wild.cuda())
    b = op.forward(lp.cuda(), old.cuda(), adv, wild.clamp(0, n).cuda())
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n", [1000, 50000])
def test_policy_views_at_odd_addresses(n):
    """Token arrays that begin at any element (slices of a longer batch)."""
    g = torch.Generator().manual_seed(3)
    lp, old, ref = (t.cuda() for t in _tokens(g, n + 3, "f32"))
    mask = (torch.rand(n + 3, generator=g) < 0.6).to(torch.uint8).cuda()
    offs = _offsets(g, 6, n).cuda()
    adv = torch.randn(6, generator=g).cuda()
    op = rece.PolicyLoss(n, 6, kl_coef=0.1, reduction="sequence")
    a = op.forward(lp[3:], old[3:], adv, offs, ref_logp=ref[3:], mask=mask[3:])
    b = op.forward(lp[3:].clone(), old[3:].clone(), adv, offs, ref_logp=ref[3:].clone(), mask=mask[3:].clone())
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)


PREF = [
    # groups, rejected (max), tokens, dtype, kind, smoothing, average, masked, margin, reference
    (1, 1, 2, "f32", "sigmoid", 0.0, False, False, 0.0, True),
    (1, 1, 3000, "f32", "sigmoid", 0.1, False, True, 0.5, True),
    (5, 1, 300, "f32", "ipo", 0.0, True, True, 0.0, True),
    (40, 3, 200, "bf16", "hinge", 0.0, False, True, 0.0, True),
    (40, 3, 200, "f32", "softmax", 0.0, False, False, 0.2, False),
    (300, 7, 20000, "bf16", "softmax", 0.0, True, True, 0.0, True),
    (2, 900, 5000, "f32", "softmax", 0.0, False, True, 0.0, True),
    (2, 900, 90000, "f32", "sigmoid", 0.2, False, True, 0.0, True),
    (64, 1, 128, "f32", "sigmoid", 0.0, False, False, 0.0, False),
    (3, 30, 40, "f32", "ipo", 0.0, False, False, 0.1, True),
]


@pytest.mark.parametrize("G,K,n,dtype,kind,smoothing,average,masked,margin,with_ref", PREF)
def test_preference_against_plain(G, K, n, dtype, kind, smoothing, average, masked, margin, with_ref):
    g = torch.Generator().manual_seed(G * 31 + n)
    sizes = torch.randint(0, K + 2, (G,), generator=g)
    sizes[0] = K + 1
    lead = 2
    goffs = torch.cat([torch.tensor([lead]), lead + sizes.cumsum(0)]).to(torch.int32)
    n_seq = int(goffs[-1]) + 3
    lp, ref, _ = _tokens(g, n, dtype)
    if not with_ref:
        ref = None
    offs = _offsets(g, n_seq, n, lead=min(1, n - 1), trail=min(1, n - 1))
    mask = (torch.rand(n, generator=g) < 0.7).to(torch.uint8) if masked else None
    if masked:
        lp = lp.clone()
        lp[mask == 0] = float("nan")
    beta = 0.25
    cfg = dict(beta=beta, kind=kind, smoothing=smoothing, average=average, margin=margin)
    print(f"[gpu] preference G={G} K={K} n={n} {dtype} {kind} average={average} masked={masked}", flush=True)
    op = rece.PreferenceLoss(n, n_seq, G, beta=beta, kind=kind, label_smoothing=smoothing, margin=margin, average=average,
                             dtype=dtype)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    dloss = torch.full((1,), 3.0, device="cuda")
    loss, loss_pg, rewards, dlp = op.forward(cu(lp), cu(ref), cu(offs), cu(goffs), mask=cu(mask), dloss=dloss)
    # the reference in the library's own constants (float32 options)
    f = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    cfg.update(beta=f(beta), smoothing=f(smoothing), margin=f(margin))
    wl, wpg, wr, wg = R.preference(lp, ref, offs, goffs, cfg, mask)
    # token ratios: one float32 difference (U32 of up to 8 each), summed in float64
    seq = R.seq_of_tokens(offs, n)
    on = (seq >= 0) & ((mask != 0) if mask is not None else torch.ones(n, dtype=torch.bool))
    count = torch.zeros(n_seq, dtype=torch.float64).index_add_(0, seq[on], torch.ones(int(on.sum()), dtype=torch.float64))
    eh = 8 * R.U32 * (torch.ones_like(count) if average else count) * (0.0 if ref is None else 1.0) + 1e-13
    assert bool(((rewards.cpu().double() - wr).abs() <= beta * eh + 2 * R.U32 * wr.abs()).all())
    o = goffs.long()
    # loss by z: slope at most 1 (sigmoid, hinge, softmax), 2 |v| / beta (ipo); second derivative at
    # most 1, for ipo 2 / beta^2, none for hinge away from its corner
    hh = wr / cfg["beta"]
    big = 4.0 * R.U32
    for q in range(G):
        lo, hi = int(o[q]), int(o[q + 1])
        ez = beta * 2 * float(eh[lo:hi].max()) if hi > lo else 0.0
        slope = 1.0
        if kind == "ipo" and hi - lo >= 2:
            slope = 2 * float(((hh[lo] - hh[lo + 1:hi]).abs() + (margin + 0.5) / beta).max()) / beta
        assert abs(float(loss_pg[q]) - float(wpg[q])) <= slope * ez + big * abs(float(wpg[q])), q
    assert abs(float(loss) - wl) <= float((loss_pg.cpu().double() - wpg).abs().mean()) + 2 * R.U32 * float(wpg.abs().mean())
    second = {"ipo": 2 / beta ** 2, "hinge": 0.0}.get(kind, 1.0)
    ez = beta * 2 * float(eh.max())
    u = R.U[DT[dtype]]
    tol = beta * second * ez / G + (u + 16 * R.U32) * wg.abs()
    assert bool(((dlp.cpu().double() - 3 * wg).abs() <= 3 * tol + 1e-12).all())
    assert bool((dlp.cpu()[~on] == 0).all())
    again = op.forward(cu(lp), cu(ref), cu(offs), cu(goffs), mask=cu(mask), dloss=dloss)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, loss_pg, rewards, dlp)))


def test_preference_groups_outside_are_clamped():
    g = torch.Generator().manual_seed(6)
    lp, ref, _ = (t.cuda() for t in _tokens(g, 200, "f32"))
    offs = _offsets(g, 12, 200).cuda()
    goffs = torch.tensor([-4, 3, 7, 40], dtype=torch.int32)
    op = rece.PreferenceLoss(200, 12, 3)
    a = op.forward(lp, ref, offs, goffs.cuda())
    b = op.forward(lp, ref, offs, goffs.clamp(0, 12).cuda())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_capture_replay():
    n, n_seq, G = 20000, 120, 40
    g = torch.Generator().manual_seed(9)
    lp, old, ref = (t.cuda() for t in _tokens(g, n, "f32"))
    offs = _offsets(g, n_seq, n).cuda()
    goffs = torch.arange(0, n_seq + 1, 3, dtype=torch.int32).cuda()
    adv = torch.randn(n_seq, generator=g).cuda()
    mask = (torch.rand(n, generator=g) < 0.8).cuda()
    pol = rece.PolicyLoss(n, n_seq, kl_coef=0.1, reduction="sequence")
    pref = rece.PreferenceLoss(n, n_seq, G, kind="softmax")

    def both():
        return pol.forward(lp, old, adv, offs, ref_logp=ref, mask=mask)[:3] + pref.forward(lp, ref, offs, goffs, mask=mask)

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = both()
    for r in range(3):
        for t in got:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), r
        assert all(torch.equal(a, b) for a, b in zip(both(), want))


def test_a_policy_update_and_a_preference_update_end_to_end():
    """embed -> (a linear model) -> log_probs -> policy / preference loss -> gradients of the model and of
    the item table, which is used twice (input rows and output logits), against float64 autograd."""
    n_seq, per, C, d = 12, 20, 700, 64
    n = n_seq * per
    g = torch.Generator().manual_seed(21)
    table = torch.randn(C, d, generator=g) * d ** -0.25
    W = torch.eye(d) + 0.1 * torch.randn(d, d, generator=g)
    inp = torch.randint(0, C, (n,), generator=g).to(torch.int32)
    act = torch.randint(0, C, (n,), generator=g).to(torch.int32)
    act[::7] = -1
    offs = torch.arange(0, n + 1, per, dtype=torch.int32)
    goffs = torch.arange(0, n_seq + 1, 3, dtype=torch.int32)
    adv = torch.randn(n_seq, generator=g)
    mask = (act >= 0).to(torch.uint8)
    emb = rece.ItemEmbedding(n, C, d, dtype="f32", scale=0.5)
    lpo = rece.LogProb(n, C, d, dtype="f32", entropy=True)
    pol = rece.PolicyLoss(n, n_seq, kl_coef=0.1, entropy_coef=0.05)
    prf = rece.PreferenceLoss(n, n_seq, n_seq // 3, beta=0.3, kind="softmax")
    ref = -6.0 - torch.rand(n, generator=g)
    old = ref + 0.1

    def plain(kind):
        t, w = table.double().requires_grad_(True), W.double().requires_grad_(True)
        X = (t[inp.long()] * 0.5) @ w
        logq = torch.log_softmax(X @ t.T, 1)
        on = torch.nonzero(act >= 0)[:, 0]
        lp, H = logq[on, act[on].long()], -(logq.exp() * logq).sum(1)[on]
        seq = on // per
        if kind == "policy":
            r, A = (lp - old.double()[on]).exp(), adv.double()[seq]
            u = ref.double()[on] - lp
            loss = (-torch.minimum(r * A, r.clamp(0.8, 1.2) * A) + 0.1 * (u.exp() - u - 1) - 0.05 * H).mean()
        else:
            h = torch.zeros(n_seq, dtype=torch.float64).index_add(0, seq, lp - ref.double()[on]).view(-1, 3)
            z = 0.3 * (h[:, :1] - h[:, 1:])
            loss = torch.log1p((-z).exp().sum(1)).mean()
        loss.backward()
        return float(loss), t.grad, w.grad

    for kind in ("policy", "preference"):
        t, w = table.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
        X = rece.embed(t, inp.cuda(), emb) @ w
        lp, H = rece.log_probs(X, t, act.cuda(), lpo)
        if kind == "policy":
            loss, _ = rece.policy_loss(lp, old.cuda(), adv.cuda(), offs.cuda(), pol, ref_logp=ref.cuda(), entropy=H,
                                       mask=mask.cuda())
        else:
            loss, _, _ = rece.preference_loss(lp, ref.cuda(), offs.cuda(), goffs.cuda(), prf, mask=mask.cuda())
        loss.backward()
        wl, wt, ww = plain(kind)
        # a chain of float32 sums of up to C terms: 2^-24 each, so 1e-4 of the largest gradient is ample
        assert abs(float(loss) - wl) <= 1e-4 * max(abs(wl), 1.0)
        for a, b in ((t.grad, wt), (w.grad, ww)):
            assert float((a.cpu().double() - b).abs().max()) <= 1e-4 * float(b.abs().max())
