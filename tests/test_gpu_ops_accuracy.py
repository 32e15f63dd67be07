"""How near the operators come to their 64-bit forms where float32 or bf16 intermediates would show."""
import numpy as np
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R
import test_gpu_logprob as TL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s,C,d,entropy", [
    (8, 2000, 64, False), (8, 2000, 64, True), (70, 9, 32, False), (300, 12, 128, True), (300, 12, 256, False),
    (9, 700, 256, True), (70, 400, 128, False), (600, 40, 64, False), (40, 30000, 64, False),
])
def test_logprob_bf16_gradients_round_the_results_alone(s, C, d, entropy):
    """bf16 gradients are the float32 ones rounded, but for 2^-16 of each weight (two bf16 terms, each off by at most
    half a step: 2^-8 of 2^-8).  Few positions or few items: results much smaller than their terms, where weights
    rounded to bf16 would be off by up to 13 times the bound."""
    X, Y, ids, dlogp, dent, bad = TL._case(s, C, d, "bf16", seed=s + C + d, pad=0.1, peak=0.5)
    if not entropy:
        dent = None
    print(f"[gpu] logprob bf16 gradients s={s} C={C} d={d} entropy={entropy}", flush=True)
    _, _, dX, dY = TL._run(X, Y, ids, dlogp, dent, 0.9, entropy, True)
    w = R.logprob(X, Y, ids, 0.9, dlogp, dent)
    assert bool((dX[bad] == 0).all())
    for name, got in (("dX", dX), ("dY", dY)):
        assert got.dtype == torch.bfloat16
        bound = w["p_" + name] + 2.0 ** -8 * w["b_" + name]
        bound = bound + R.U[torch.bfloat16] * (w[name].abs() + bound) + 1e-30
        err = (got.double() - w[name]).abs()
        assert bool((err <= bound).all()), (name, float((err / bound).max()))


@pytest.mark.parametrize("n", [900, 30000])
@pytest.mark.parametrize("size", [1e-6, 1e-4, 1e-2, 0.3, 0.999, 1.5, 4.0])
def test_policy_kl_near_its_reference(n, size):
    """KL term and its gradient relative to their own size, however near the policy is to its reference.  Up to |u| = 1
    the differences are exact (both within a factor of two); a series of ten terms by Horner's rule leaves 5 roundings
    of its value, its two products and the mean 3; its gradient u + kl 6, the weight and the coefficient's products 4.
    Beyond, e^u is off by 4 roundings: at most 19 of kl and 8 of the gradient."""
    g = torch.Generator().manual_seed(n)
    lp = -2.0 - torch.rand(n, generator=g)
    sign = torch.where(torch.rand(n, generator=g) < 0.5, -1.0, 1.0)
    ref = lp + sign * size * (0.5 + 0.5 * torch.rand(n, generator=g))
    u = ref.double() - lp.double()
    print(f"[gpu] policy kl n={n} size={size}", flush=True)
    for reduction in ("token", "sequence"):
        op = rece.PolicyLoss(n, 1, kl_coef=0.5, reduction=reduction)
        loss, stats, dlp, _ = op.forward(lp.cuda(), lp.cuda(), torch.zeros(1, device="cuda"),
                                         torch.tensor([0, n], dtype=torch.int32, device="cuda"), ref_logp=ref.cuda())
        kl = float((torch.expm1(u) - u).mean()) if size > 0.2 else float((u * u * (0.5 + u / 6 + u * u / 24 + u ** 3 / 120)).mean())
        most = (10 if size < 1 else 24) * R.U32 + (2e-9 if size <= 1e-2 else 0.0 if size > 1 else 1e-12)
        assert float(stats[1]) > 0 and abs(float(stats[1]) - kl) <= most * kl
        assert abs(float(loss) - 0.5 * kl) <= (most + 4 * R.U32) * 0.5 * kl
        want = -0.5 * torch.expm1(u) / n
        assert bool(((dlp.cpu().double() - want).abs() <= 13 * R.U32 * want.abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [2000, 40000])
def test_policy_kl_of_a_policy_that_is_its_reference(n, dtype):
    lp = (-3.0 * torch.rand(n, generator=torch.Generator().manual_seed(1))).to(TL.DT[dtype]).cuda()
    op = rece.PolicyLoss(n, 1, kl_coef=0.5, dtype=dtype)
    loss, stats, dlp, _ = op.forward(lp, lp, torch.zeros(1, device="cuda"),
                                     torch.tensor([0, n], dtype=torch.int32, device="cuda"), ref_logp=lp)
    assert float(loss) == 0.0 and float(stats[1]) == 0.0 and not bool(dlp.any())


@pytest.mark.parametrize("n", [4000, 40000])
def test_policy_clips_on_the_right_side_with_old_log_probabilities(n):
    """Log-probabilities near 0 and old ones a few steps around the bounds: their float32 difference is rounded, the
    side of the bound is that of the difference of the values themselves (64 bits hold it)."""
    g = np.random.default_rng(n)
    low = high = float(np.float32(0.2))
    half = n // 2
    lp = -g.uniform(1e-4, 0.05, n).astype(np.float32)
    lp[:half] -= np.float32(0.25)   # a ratio below 1 - low: the old one is the one near 0
    bound = np.where(np.arange(n) < half, np.log1p(-low), np.log1p(high))
    old = (lp.astype(np.float64) - bound).astype(np.float32)
    old = (old.view(np.int32) + g.integers(-2, 3, n, dtype=np.int32)).view(np.float32)
    diff = lp.astype(np.float64) - old.astype(np.float64)
    clipped = torch.from_numpy(np.where(np.arange(n) < half, diff < bound, diff > bound))
    assert 0.2 * n < int(clipped.sum()) < 0.8 * n and float(np.abs(diff - bound).min()) > 1e-14
    rounded = (lp - old).astype(np.float64)
    assert (np.where(np.arange(n) < half, rounded < bound, rounded > bound) != clipped.numpy()).sum() > n // 100
    A = torch.cat([torch.full((half,), -1.0), torch.ones(n - half)]).cuda()
    op = rece.PolicyLoss(n, 1, clip_low=0.2, clip_high=0.2, token_advantage=True)
    _, stats, dlp, _ = op.forward(torch.from_numpy(lp).cuda(), torch.from_numpy(old).cuda(), A,
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    assert torch.equal(dlp.cpu() == 0, clipped)
    assert abs(float(stats[3]) - float(clipped.double().mean())) <= R.U32


def test_policy_without_a_lower_bound():
    """clip_low = 1 bounds nothing: ratios down to 0 pass with a negative advantage."""
    lp = torch.tensor([-1.0, -50.0, -300.0, float("-inf")]).repeat(2500)
    for n in (4, 10000):
        op = rece.PolicyLoss(n, 1, clip_low=1.0, clip_high=0.2)
        _, stats, dlp, _ = op.forward(lp[:n].cuda(), torch.zeros(n, device="cuda"), torch.tensor([-1.0], device="cuda"),
                                      torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        assert float(stats[3]) == 0.0
        want = lp[:n].double().exp() / n
        assert bool(((dlp.cpu().double() - want).abs() <= 9 * R.U32 * want + 1e-35).all())
    # and a ratio of 0 is below any other
    op = rece.PolicyLoss(4, 1, clip_low=0.9, clip_high=0.2)
    _, stats, dlp, _ = op.forward(lp[:4].cuda(), torch.zeros(4, device="cuda"), torch.tensor([-1.0], device="cuda"),
                                  torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    assert float(stats[3]) == 0.75 and (dlp == 0).tolist() == [False, True, True, True]


@pytest.mark.parametrize("n", [16, 8000, 40000, 300000])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("lead", [0, 1])
def test_policy_sums_lose_nothing(n, reduction, lead):
    """Terms that cancel across neighbouring tokens (advantages 1e8, 1, -1e8, 1, ratios of 1): the sums are exact in
    64 bits, so loss and mean are off by their own rounding and that of a 64-bit weight."""
    A = torch.tensor([1e8, 1.0, -1e8, 1.0]).repeat(n // 4)
    lp = torch.full((n + lead,), -1.0, device="cuda")[lead:]
    op = rece.PolicyLoss(n, 2, reduction=reduction, token_advantage=True)
    offs = torch.tensor([0, n // 4, n], dtype=torch.int32, device="cuda")
    loss, stats, _, _ = op.forward(lp, lp, A.cuda(), offs)
    # the plain sum is one of whole numbers below 2^53.  Weighted: a thread's 16 additions and some ten levels of joins,
    # each off by 2^-53 of at most 1e8 times the number of tokens so far, weights of at most 2 / n: below 60 of them
    most = 64 * 2.0 ** -53 * 1e8 + R.U32
    assert abs(float(loss) + 0.5) <= most and abs(float(stats[0]) + 0.5) <= most


@pytest.mark.parametrize("n,n_seq", [(7000, 3), (50001, 3), (400003, 7), (50001, 5000)])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_loss_is_off_by_its_own_rounding(n, n_seq, reduction):
    """Ratios of 1 leave no rounding in the terms: the loss is the float64 mean of the advantages, rounded once."""
    g = torch.Generator().manual_seed(n)
    cut = torch.sort(torch.randint(0, n + 1, (n_seq + 1,), generator=g)).values
    cut[0], cut[-1] = 0, n
    mask = torch.rand(n, generator=g) < 0.7
    A = 1.0 + torch.rand(n, generator=g)
    lp = torch.full((n,), -2.0, device="cuda")
    op = rece.PolicyLoss(n, n_seq, reduction=reduction, token_advantage=True)
    loss, stats, _, _ = op.forward(lp, lp, A.cuda(), cut.to(torch.int32).cuda(), mask=mask.cuda())
    seq = R.seq_of_tokens(cut, n)
    on = mask & (seq >= 0)
    count = torch.zeros(n_seq, dtype=torch.float64).index_add_(0, seq[on], torch.ones(int(on.sum()), dtype=torch.float64))
    w = 1.0 / on.sum().double() if reduction == "token" else 1.0 / (count[seq[on]] * (count > 0).sum())
    want = -float((A[on].double() * w).sum())
    assert abs(float(loss) - want) <= (R.U32 + 1e-12) * abs(want)
    assert abs(float(stats[0]) + float(A[on].double().mean())) <= (R.U32 + 1e-12) * abs(want) * 1.5


def _token_pairs(G, lens, seed):
    """Sequences of the given lengths in turn, two a group; values in 1/64 steps, so that float32 holds their
    differences and float64 their sums exactly."""
    g = torch.Generator().manual_seed(seed)
    count = torch.tensor([lens[i % len(lens)] for i in range(2 * G)])
    offs = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)])
    lp = -torch.randint(1, 512, (int(offs[-1]),), generator=g) / 64.0
    return lp, offs.to(torch.int32), (torch.arange(G + 1) * 2).to(torch.int32)


def test_preference_loss_is_off_by_its_own_rounding():
    """The mean is taken of the groups' float64 losses, not of their roundings: off by half a step however they lie
    (among 300 draws of three groups, roundings of the three that add up to more are common)."""
    for seed in range(300):
        lp, offs, goffs = _token_pairs(3, (1, 2), seed)
        cfg = dict(beta=0.25, kind="sigmoid", smoothing=0.0, average=False, margin=0.0)
        op = rece.PreferenceLoss(lp.numel(), 6, 3, beta=0.25)
        loss, pg, _, _ = op.forward(lp.cuda(), None, offs.cuda(), goffs.cuda())
        want, want_pg, _, _ = R.preference(lp, None, offs, goffs, cfg)
        assert abs(float(loss) - want) <= (R.U32 + 1e-12) * want, seed
        assert bool(((pg.cpu().double() - want_pg).abs() <= (R.U32 + 1e-12) * want_pg).all()), seed


@pytest.mark.parametrize("G,lens", [(40, (3, 7, 5)), (40, (90, 70, 110)), (3000, (3, 2, 3)), (3000, (11, 7, 13)), (30, (1, 3))])
def test_preference_average_gradient_is_off_by_its_own_rounding(G, lens):
    """The share 1 / tokens of an averaged sequence is not rounded before the product."""
    lp, offs, goffs = _token_pairs(G, lens, 5)
    cfg = dict(beta=0.5, kind="sigmoid", smoothing=0.25, average=True, margin=0.0)
    op = rece.PreferenceLoss(lp.numel(), 2 * G, G, beta=0.5, label_smoothing=0.25, average=True)
    _, _, _, dlp = op.forward(lp.cuda(), None, offs.cuda(), goffs.cuda())
    want = R.preference(lp, None, offs, goffs, cfg)[3]
    assert bool(((dlp.cpu().double() - want).abs() <= (R.U32 + 1e-12) * want.abs() + 1e-17).all())


def test_preference_average_gradient_of_a_large_group():
    """More members than the workgroup's own memory holds: their shares lie in the workspace."""
    m, lens = 700, (3, 7, 1, 5)
    count = torch.tensor([lens[i % 4] for i in range(m)])
    offs = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)]).to(torch.int32)
    lp = -torch.randint(1, 512, (int(offs[-1]),), generator=torch.Generator().manual_seed(2)) / 64.0
    goffs = torch.tensor([0, m], dtype=torch.int32)
    cfg = dict(beta=0.5, kind="softmax", smoothing=0.0, average=True, margin=0.0)
    op = rece.PreferenceLoss(lp.numel(), m, 1, beta=0.5, kind="softmax", average=True)
    loss, _, _, dlp = op.forward(lp.cuda(), None, offs.cuda(), goffs.cuda())
    want, _, _, grad = R.preference(lp, None, offs, goffs, cfg)
    assert abs(float(loss) - want) <= (R.U32 + 1e-12) * want
    assert bool(((dlp.cpu().double() - grad).abs() <= (R.U32 + 1e-12) * grad.abs() + 1e-17).all())


def _near_one(s, C, d, dtype, seed):
    """Positions whose own item has a probability from 0.99 to 1 - 1e-6, each an item of its own."""
    g = torch.Generator().manual_seed(seed)
    Y = torch.randn(C, d, generator=g) * d ** -0.25
    ids = torch.randperm(C, generator=g)[:s].to(torch.int32)
    a = Y[ids.long()]
    rest = torch.randn(s, d, generator=g) * 0.3 * d ** -0.25
    X = a / (a * a).sum(1, keepdim=True) * torch.linspace(9.0, 25.0, s)[:, None] + rest
    X, Y = X.to(TL.DT[dtype]), Y.to(TL.DT[dtype])
    left = 1.0 - torch.softmax(X.double() @ Y.double().T, 1)[torch.arange(s), ids.long()]
    keep = (left < 0.01) & (left > 1e-6)
    assert int(keep.sum()) > s // 3 and float(left[keep].min()) < 1e-5
    ids[~keep] = -1
    return X, Y, ids, torch.randn(s, generator=g) / s, torch.randn(s, generator=g) / s * 0.1


@pytest.mark.parametrize("s,C,d", [(60, 90, 64), (150, 160, 128), (150, 160, 32), (100, 130, 256)])
@pytest.mark.parametrize("dtype,bf16_grads", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("entropy", [False, True])
def test_logprob_near_certainty(s, C, d, dtype, bf16_grads, entropy):
    """Where p is near 1: log p is off relative to 1 - p, and so is the own item's weight g (1 - p), but for the
    roundings of float32 sums that its term and its row pass through (one per 16 rows of the products and per join)."""
    X, Y, ids, dlogp, dent = _near_one(s, C, d, dtype, seed=s + d)
    if not entropy:
        dent = None
    print(f"[gpu] logprob near 1 s={s} C={C} d={d} {dtype} bf16_grads={bf16_grads} entropy={entropy}", flush=True)
    logp, _, dX, dY = TL._run(X, Y, ids, dlogp, dent, 1.0, entropy, bf16_grads)
    w = R.logprob(X, Y, ids, 1.0, dlogp, dent)
    on = ids >= 0
    k = torch.arange(int(on.sum()))
    a, Xk, Yd = ids[on].long(), X.double()[on], Y.double()
    L = Xk @ Yd.T
    logq = torch.log_softmax(L, 1)
    q = logq.exp()
    left = -torch.expm1(logq[k, a])
    # the bounds of R.logprob for logits, exponentials and their sum, relative to what they scale
    ex = (d + 4) * R.U32 * (Xk.abs() @ Yd.abs().T).amax(1)
    elog = 2 * ex + (16 + C / 32 + 112 + 8 * L.abs().amax(1)) * R.U32
    rel = 2 * ex + elog + 8 * R.U32
    # log p = -log1p((1 - p) / p), (1 - p) / p the others' sum over the own term.  The others' sum is the float32 sum of
    # all less the own term, and nearly all of that sum is the own term: each addition after it (at most 16 of its
    # block, one per block, 4 of lane halves and parts) rounds by U32 of it, and so does each product and difference
    # that takes it out (3), whatever is left.
    most = (rel + 4 * R.U32) * left + (16 + C / 32 + 4 + 3) * R.U32
    assert bool(((logp.double()[on] - logq[k, a]).abs() <= 1.02 * most).all())
    gk = dlogp.double()[on].abs()
    hk = dent.double()[on].abs() if entropy else torch.zeros_like(gk)
    H = -(q * logq).sum(1)
    size = q * (gk[:, None] + hk[:, None] * (logq.abs() + H[:, None]))
    size[k, a] = gk * left + hk * q[k, a] * (logq[k, a].abs() + H)
    off = size * (rel[:, None] + (2.0 ** -16 if bf16_grads else 0.0)) + q * (hk * w["e_entropy"][on])[:, None]
    hot = torch.zeros_like(q)
    hot[k, a] = gk
    steps = (C + s) / 16 + 24
    u = R.U[torch.bfloat16] if bf16_grads else R.U32
    for got, want, bound in ((dX[on], w["dX"][on], off @ Yd.abs() + steps * R.U32 * ((hot + size) @ Yd.abs())),
                             (dY, w["dY"], off.T @ Xk.abs() + steps * R.U32 * ((hot + size).T @ Xk.abs()))):
        bound = bound + u * (want.abs() + bound) + 1e-30
        err = (got.double() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())


def _long_among_short(G, members, short, long, seed):
    """Groups of sequences of `short` tokens, a few of `long` tokens, and one each before and behind the groups."""
    g = torch.Generator().manual_seed(seed)
    n_seq = G * members + 2
    lens = torch.full((n_seq,), short)
    at = torch.randperm(n_seq - 2, generator=g)[:5] + 1
    lens[at] = torch.tensor([long, long - 1, long // 2 + 3, 33, 1025])
    lens[0], lens[-1] = long // 3, long + 5
    offs = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]) + 3
    n = int(offs[-1]) + 2
    lp, ref = (-4.0 * torch.rand(n, generator=g) for _ in range(2))
    return lp, ref, offs.to(torch.int32), (1 + torch.arange(G + 1) * members).to(torch.int32), torch.rand(n, generator=g) < 0.8


@pytest.mark.parametrize("G,members,short", [(3000, 2, 1), (3000, 2, 9), (9000, 4, 1), (9000, 3, 6), (60, 5, 1), (60, 3, 7), (60, 90, 5)])
@pytest.mark.parametrize("kind,average", [("sigmoid", True), ("softmax", False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lead", [0, 1])
def test_preference_long_sequences_among_short_ones(G, members, short, kind, average, dtype, lead):
    """Lanes per sequence go by the mean length; what is left of a longer sequence the whole wave takes.  Every ratio of
    float32 or bf16 tokens is off by U32 of at most 4 in its difference, its sum is float64; the gradient is beta times a
    slope of at most 1 / G whose own slope by h is at most beta."""
    dt = TL.DT[dtype]
    long = 3000 if short < 4 else 6000
    lp, ref, offs, goffs, mask = _long_among_short(G, members, short, long, G + short)
    lp, ref = lp.to(dt), ref.to(dt)
    n, n_seq = lp.numel(), offs.numel() - 1
    beta = 0.125
    op = rece.PreferenceLoss(n, n_seq, G, beta=beta, kind=kind, average=average, dtype=dtype)
    put = lambda t: torch.cat([t[:1].expand(lead), t]).cuda()[lead:]  # noqa: E731
    print(f"[gpu] preference long G={G} members={members} short={short} {kind} {dtype} lead={lead}", flush=True)
    poison = torch.full((), float("nan"), dtype=dt)
    loss, pg, rewards, dlp = op.forward(put(torch.where(mask, lp, poison)), put(ref), offs.cuda(), goffs.cuda(), mask=put(mask))
    # the float64 form over sums per sequence (thousands of groups: without the loop of the plain one)
    seq = torch.repeat_interleave(torch.arange(n_seq), offs.long().diff())
    inside = slice(int(offs[0]), int(offs[-1]))
    ratio = torch.where(mask, lp.double() - ref.double(), 0.0)[inside]
    zero = torch.zeros(n_seq, dtype=torch.float64)
    count = zero.index_add(0, seq, mask[inside].double())
    h = zero.index_add(0, seq, ratio)
    eh = 4 * R.U32 * count + 1e-12
    if average:
        h, eh = h / count.clamp(min=1), eh / count.clamp(min=1)
    assert bool(((rewards.cpu().double() - beta * h).abs() <= beta * eh + 1.01 * R.U32 * beta * h.abs()).all())
    hg, eg = h[1:-1].view(G, members), eh[1:-1].view(G, members)
    z, ez = beta * (hg[:, :1] - hg[:, 1:]), beta * (eg[:, :1] + eg[:, 1:])
    if kind == "softmax":
        tot = 1.0 + (-z).exp().sum(1)
        want_pg, dz = tot.log(), -(-z).exp() / tot[:, None]
    else:
        want_pg = torch.nn.functional.softplus(-z, threshold=1e9).mean(1)
        dz = (torch.sigmoid(z) - 1.0) / (members - 1)
    assert bool(((pg.cpu().double() - want_pg).abs() <= ez.sum(1) + 1.01 * R.U32 * want_pg).all())
    assert abs(float(loss) - float(want_pg.mean())) <= float(ez.sum(1).mean()) + 1.01 * R.U32 * float(want_pg.mean())
    dh, edh = zero.clone(), zero.clone()
    dh[1:-1] = torch.cat([dz.sum(1, keepdim=True), -dz], 1).flatten() * beta / G
    slope = ez.sum(1, keepdim=True) * beta / G   # each derivative moves by at most the sum of the z's errors
    edh[1:-1] = slope.expand(G, members).flatten()
    if average:
        dh, edh = dh / count.clamp(min=1), edh / count.clamp(min=1)
    want, err = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    want[inside], err[inside] = dh[seq], edh[seq]
    want = torch.where(mask, want, 0.0)
    got = dlp.cpu().double()
    assert bool(((got - want).abs() <= err + 1.01 * R.U[dt] * (want.abs() + err)).all())
    assert not bool(got[~mask].any()) and not bool(got[:int(offs[1])].any()) and not bool(got[int(offs[-2]):].any())


@pytest.mark.parametrize("G", [200, 9000])
@pytest.mark.parametrize("kind,members", [("sigmoid", 2), ("sigmoid", 4), ("softmax", 2), ("softmax", 4)])
def test_preference_pairs_that_are_well_apart(G, kind, members):
    """z from 1 to 80: loss and gradient fall to e^-80 and stay exact to their own rounding (values in steps of 1/64, so
    z is exact, and e^-z is off by 80 steps of 2^-53)."""
    g = torch.Generator().manual_seed(G)
    h = -40.0 * torch.rand(G, members, generator=g)
    h[:, 0] = 1.0 + 39.0 * torch.rand(G, generator=g)
    h = (h * 64).round() / 64
    n = G * members
    op = rece.PreferenceLoss(n, n, G, beta=1.0, kind=kind)
    loss, pg, _, dlp = op.forward(h.flatten().cuda(), None, torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                                  (torch.arange(G + 1) * members).to(torch.int32).cuda())
    z = h[:, :1].double() - h[:, 1:].double()
    if kind == "softmax":
        e = (-z).exp()
        want, dz = torch.log1p(e.sum(1)), -e / (1.0 + e.sum(1, keepdim=True))
    else:
        want, dz = torch.log1p((-z).exp()).mean(1), -1.0 / (1.0 + z.exp()) / (members - 1)
    grad = torch.cat([dz.sum(1, keepdim=True), -dz], 1) / G
    u = R.U32 + 1e-13
    assert bool(((pg.cpu().double() - want).abs() <= u * want).all())
    assert abs(float(loss) - float(want.mean())) <= u * float(want.mean())
    # (e^-80 / 9,000 lies below the normal float32 numbers)
    assert bool(((dlp.cpu().double().view(G, members) - grad).abs() <= u * grad.abs() + 2.0 ** -126).all())


@pytest.mark.parametrize("per", [1, 2, 9])
@pytest.mark.parametrize("kind", ["sigmoid", "ipo", "hinge", "softmax"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_large_groups_among_many_small_ones(per, kind, average):
    """Groups of 64, 65, 200 and 3,000 members among 9,000 pairs.  Tokens in steps of 1/64 and no reference, so that every
    h is exact in 64 bits: results are off by their own rounding, but for 64-bit sums of up to 3,000 terms (and what
    lies below the normal float32 numbers: z reaches 300)."""
    G = 9000
    size = torch.full((G,), 2)
    size[[5, 6, 7000, G - 1, 100]] = torch.tensor([64, 65, 3000, 200, 0])
    goffs = torch.cat([torch.zeros(1, dtype=torch.long), size.cumsum(0)])
    n_seq = int(goffs[-1])
    lens = torch.full((n_seq,), per)
    lens[::5] += 1
    lens[20:3000:700] = 600
    offs = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    n = int(offs[-1])
    lp = -torch.randint(1, 512, (n,), generator=torch.Generator().manual_seed(per)) / 64.0
    beta = 0.125
    op = rece.PreferenceLoss(n, n_seq, G, beta=beta, kind=kind, average=average, margin=0.25)
    print(f"[gpu] preference large groups {kind} per={per} average={average}", flush=True)
    loss, pg, rewards, dlp = op.forward(lp.cuda(), None, offs.to(torch.int32).cuda(), goffs.to(torch.int32).cuda())
    seq, grp = torch.repeat_interleave(torch.arange(n_seq), lens), torch.repeat_interleave(torch.arange(G), size)
    x = lp.double().requires_grad_(True)
    h = torch.zeros(n_seq, dtype=torch.float64).index_add(0, seq, x)
    if average:
        h = h / lens
    first = goffs[:-1][grp]
    other = torch.arange(n_seq) > first
    z = (beta * (h[first] - h) - 0.25)[other]
    per_group = lambda v: torch.zeros(G, dtype=torch.float64).index_add(0, grp[other], v)  # noqa: E731
    if kind == "softmax":
        want = torch.log1p(per_group((-z).exp()))
    else:
        each = {"sigmoid": lambda: -torch.nn.functional.logsigmoid(z), "hinge": lambda: torch.relu(1 - z),
                "ipo": lambda: (z / beta - 0.5 / beta) ** 2}[kind]()
        want = per_group(each) / (size - 1).clamp(min=1)
    want.mean().backward()
    tiny = 3000 * 2.0 ** -52
    want = want.detach()
    assert bool(((pg.cpu().double() - want).abs() <= (R.U32 + tiny) * want + 2.0 ** -126).all())
    assert abs(float(loss) - float(want.mean())) <= (R.U32 + tiny) * float(want.mean())
    assert bool(((rewards.cpu().double() - beta * h.detach()).abs() <= (R.U32 + tiny) * beta * h.detach().abs()).all())
    # the preferred one's gradient is a sum of its group's, which may cancel for ipo
    scale = torch.zeros(G, dtype=torch.float64).index_add(0, grp, torch.zeros(n_seq, dtype=torch.float64).index_add(
        0, seq, x.grad.abs()))[grp][seq]
    assert bool(((dlp.cpu().double() - x.grad).abs() <= (R.U32 + 1e-12) * x.grad.abs() + tiny * scale + 2.0 ** -126).all())


@pytest.mark.parametrize("s,C,d", [(1, 1006, 128), (2, 300, 64), (24, 1006, 32), (60, 90, 64), (150, 160, 128), (100, 130, 256)])
@pytest.mark.parametrize("dtype,bf16_grads", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("entropy", [False, True])
def test_logprob_keeps_the_digits_of_what_is_left(s, C, d, dtype, bf16_grads, entropy):
    """1 - p from 1e-2 to 1e-9: log p, entropy and the gradients are off relative to 1 - p alone.  No sum holds the own
    item's term, so nothing rounds by it: the others' sums are off by their logits, exponentials and additions (rel, as in
    R.logprob), and the own item's weight g (1 - p) - h p (log p + H) by what those leave in log p and H."""
    g = torch.Generator().manual_seed(s + C + d)
    Y = torch.randn(C, d, generator=g) * d ** -0.25
    ids = torch.randperm(C, generator=g)[:s].to(torch.int32)
    a = Y[ids.long()]
    X = a / (a * a).sum(1, keepdim=True) * torch.linspace(12.0, 24.0, s)[:, None] + \
        torch.randn(s, d, generator=g) * 0.1 * d ** -0.25
    X, Y = X.to(TL.DT[dtype]), Y.to(TL.DT[dtype])
    dlogp, dent = torch.randn(s, generator=g) / s, torch.randn(s, generator=g) / s * 0.1
    if not entropy:
        dent = None
    print(f"[gpu] logprob what is left s={s} C={C} d={d} {dtype} bf16_grads={bf16_grads} entropy={entropy}", flush=True)
    logp, ent, dX, dY = TL._run(X, Y, ids, dlogp, dent, 1.0, entropy, bf16_grads)
    Xd, Yd, k, at = X.double(), Y.double(), torch.arange(s), ids.long()
    L = Xd @ Yd.T
    far = L - L[k, at][:, None]
    e = far.exp()
    e[k, at] = 0.0
    t1 = e.sum(1)
    want = -torch.log1p(t1)
    left = t1 / (1.0 + t1)
    assert float(left.min()) < 1e-2 and float(left.max()) < 0.2
    q = (far + want[:, None]).exp()
    logq = far + want[:, None]
    H = -(q * logq).sum(1)
    mag = (Xd.abs() @ Yd.abs().T).amax(1)
    ex = (d + 4) * R.U32 * mag
    rel = 4 * ex + (16 + C / 32 + 112 + 8 * L.abs().amax(1) + 8) * R.U32
    assert bool(((logp.double() - want).abs() <= 1.02 * (rel + 4 * R.U32) * left).all())
    if entropy:
        # terms of one sign, p (-log p): p off by rel, log p by the logits' error, of a size of 1 and more but the own one's
        assert bool(((ent.double() - H).abs() <= 2.0 * (rel + 16 * R.U32) * (H + left)).all())
    gk, hk = dlogp.double(), dent.double() if entropy else torch.zeros(s, dtype=torch.float64)
    G = -q * (gk[:, None] + hk[:, None] * (logq + H[:, None]))
    G[k, at] = gk * left - hk * q[k, at] * (want + H)
    size = q * (gk.abs()[:, None] + hk.abs()[:, None] * (logq.abs() + H[:, None] + 1.0))
    size[k, at] = gk.abs() * left + 2.0 * hk.abs() * (want.abs() + H + left)
    off = size * (1.02 * rel[:, None] + 16 * R.U32 + (2.0 ** -16 if bf16_grads else 0.0))
    steps = (C + s) / 16 + 24   # additions that a result passes through, each off by U32 of at most the sum of sizes
    u = R.U[torch.bfloat16] if bf16_grads else R.U32
    for got, w, bound in ((dX, G @ Yd, (off + steps * R.U32 * size) @ Yd.abs()), (dY, G.T @ Xd, (off + steps * R.U32 * size).T @ Xd.abs())):
        bound = bound + u * (w.abs() + bound) + 1e-30
        err = (got.double() - w).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
