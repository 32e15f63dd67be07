"""The operators at sizes beyond the usual: arrays of more than 2^31 elements, sorts of many positions, millions of
groups, and values that nothing may read."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R
import test_gpu_logprob as TL

pytestmark = pytest.mark.gpu


def _need(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def test_embed_of_a_table_beyond_32_bits():
    C, d, n = 17_000_003, 128, 5000   # 2.2e9 elements
    _need(24)
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(C - 300, C, (n,), generator=g).to(torch.int32)
    ids[::3] = torch.randint(0, 300, (ids[::3].numel(),), generator=g).to(torch.int32)
    ids[::7] = -1
    table = torch.zeros(C, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(600, d, generator=g).bfloat16().cuda()
    table[:300], table[-300:] = rows[:300], rows[300:]
    op = rece.ItemEmbedding(n, C, d, scale=2.0)
    out = op.forward(table, ids.cuda())
    at = torch.where(ids < 300, ids, ids - (C - 600)).long().cuda()   # rows of `rows`
    keep = (ids >= 0).cuda()
    assert torch.equal(out, torch.where(keep[:, None], rows[at.clamp(min=0)] * 2, 0))
    del table
    dout = torch.randn(n, d, generator=g).bfloat16()
    got = op.backward(ids.cuda(), dout.cuda())
    small = torch.where(ids < 0, -1, at.cpu().to(torch.int32))
    grad, bound = R.embed_grad(small, dout, 600, 2.0)
    mine = torch.cat([got[:300], got[-300:]]).cpu().double()
    assert bool(((mine - grad).abs() <= bound).all())
    assert not bool(got[300:-300].any())


@pytest.mark.parametrize("entropy", [False, True])
def test_logprob_of_a_catalogue_beyond_32_bits(entropy):
    """2.15e9 elements of Y: the items at the end carry most of the probability."""
    s, C, d = 3, 8_400_007, 256
    _need(40)
    g = torch.Generator(device="cuda").manual_seed(2)
    Y = torch.empty(C, d, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, C, 1 << 20):
        hi = min(C, lo + (1 << 20))
        Y[lo:hi] = torch.randn(hi - lo, d, generator=g, device="cuda") * 0.25
    X = torch.randn(s, d, generator=g, device="cuda").mul_(0.25).to(torch.bfloat16)
    ids = torch.tensor([C - 1, C - 40_000, 5], dtype=torch.int32, device="cuda")
    X = (X.float() + 3.0 * Y[ids.long()].float()).to(torch.bfloat16)
    L = torch.empty(s, C, dtype=torch.float64, device="cuda")
    mag = 0.0
    for lo in range(0, C, 1 << 18):
        y = Y[lo:lo + (1 << 18)].double()
        L[:, lo:lo + (1 << 18)] = X.double() @ y.t().contiguous()
        mag = max(mag, float((X.double().abs() @ y.abs().t().contiguous()).max()))
    lse = torch.logsumexp(L, 1)
    logq = L - lse[:, None]
    want = logq[torch.arange(s), ids.long()]
    op = rece.LogProb(s, C, d, entropy=entropy, bf16_grads=True)
    logp, ent, ws = op.forward(X, Y, ids)
    # as R.logprob: a logit's d products, the reference, a sum of one term per block of 32 rows of a run and the runs'
    e = 4 * (d + 4) * R.U32 * mag + (16 + C / 32 / 256 + 1200 + 8 * float(L.abs().max())) * R.U32
    assert bool(((logp.double() - want).abs() <= e).all())
    if entropy:
        H = -(logq.exp() * logq).sum(1)
        assert bool(((ent.double() - H).abs() <= e * (float(L.max() - L.min()) + 3)).all())
    dlogp = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    dX, dY = op.backward(X, Y, ids, ws, dlogp)
    for i in range(s):   # the own items' rows, far beyond 2^31 elements: dY_a = sum over i of g_i ([own] - p_ia) X_i
        p = logq[:, int(ids[i])].exp()
        G = -dlogp.double() * p
        G[i] += dlogp[i]
        row = G @ X.double()
        bound = 2 * e * (dlogp.double().abs() * p) @ X.double().abs() + 2.0 ** -8 * row.abs() \
            + 2 * e * float(dlogp[i].abs()) * X[i].double().abs()
        assert bool(((dY[int(ids[i])].double() - row).abs() <= bound).all()), i
    rows = torch.randint(0, C, (4000,), generator=g, device="cuda")
    rows = rows[~torch.isin(rows, ids.long())]
    W = -dlogp.double()[:, None] * logq[:, rows].exp()
    want = W.t().contiguous() @ X.double()
    bound = (2 * e + 2.0 ** -15) * (W.abs().t().contiguous() @ X.double().abs()) + 2.0 ** -8 * want.abs() + 1e-30
    assert bool(((dY[rows].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("bf16_grads", [False, True])
def test_logprob_of_many_positions(bf16_grads):
    """Many positions on few items: own items in most blocks, several parts per item block."""
    s, C, d = 270_011, 37, 32
    X, Y, ids, dlogp, dent, bad = TL._case(s, C, d, "bf16", seed=4, pad=0.02, peak=1.0)
    print(f"[gpu] logprob s={s} bf16_grads={bf16_grads}", flush=True)
    logp, _, dX, dY = TL._run(X, Y, ids, dlogp, None, 1.0, False, bf16_grads)
    w = R.logprob(X, Y, ids, 1.0, dlogp, None)
    assert bool(((logp.double() - w["logp"]).abs() <= w["e_logp"]).all())
    u = R.U[torch.bfloat16] if bf16_grads else R.U32
    for name, got in (("dX", dX), ("dY", dY)):
        bound = w["p_" + name] + (2.0 ** -8 * w["b_" + name] if bf16_grads else 0.0)
        bound = bound + u * (w[name].abs() + bound) + 1e-30
        assert bool(((got.double() - w[name]).abs() <= bound).all()), name


def test_logprob_upstream_gradients_of_padding_are_not_read():
    s, C, d = 500, 300, 64
    X, Y, ids, dlogp, dent, bad = TL._case(s, C, d, "bf16", seed=6, pad=0.3, peak=1.0)
    wild = [torch.where(bad, float("nan"), t) for t in (dlogp, dent)]
    for entropy in (False, True):
        a = TL._run(X, Y, ids, dlogp, dent if entropy else None, 1.0, entropy, True)
        b = TL._run(X, Y, ids, wild[0], wild[1] if entropy else None, 1.0, entropy, True)
        assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])


@pytest.mark.parametrize("n", [600, 30000])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_advantages_that_no_token_uses_are_not_read(n, reduction):
    lp = -torch.rand(n, generator=torch.Generator().manual_seed(n))
    offs = torch.tensor([0, 0, n // 3, n // 2, n, n], dtype=torch.int32, device="cuda")
    mask = torch.ones(n, dtype=torch.uint8)
    mask[n // 3:n // 2] = 0   # of the sequences, 0 and 4 are empty and 2 counts nowhere
    adv = torch.tensor([1.0, 2.0, 3.0, -1.0, 4.0])
    wild = adv.clone()
    wild[0], wild[2], wild[4] = float("nan"), float("inf"), float("nan")
    op = rece.PolicyLoss(n, 5, reduction=reduction)
    run = lambda a: op.forward(lp.cuda(), lp.cuda() * 1.01, a.cuda(), offs, mask=mask.cuda())[:3]  # noqa: E731
    for x, y in zip(run(adv), run(wild)):
        assert torch.equal(x, y) and bool(x.isfinite().all())


def test_preference_of_millions_of_groups():
    """More groups than a launch has workgroups for along one side, a workgroup each (9 members of one token)."""
    G, m = (1 << 22) + 1001, 9
    _need(8)
    n = G * m
    g = torch.Generator(device="cuda").manual_seed(7)
    lp = -4.0 * torch.rand(n, generator=g, device="cuda")
    offs = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    goffs = torch.arange(0, n + 1, m, dtype=torch.int32, device="cuda")
    op = rece.PreferenceLoss(n, n, G, beta=0.5, kind="softmax")
    loss, pg, rewards, dlp = op.forward(lp, None, offs, goffs)
    h = lp.double().view(G, m)
    z = 0.5 * (h[:, :1] - h[:, 1:])
    tot = 1.0 + (-z).exp().sum(1)
    assert bool(((pg.double() - tot.log()).abs() <= 2 * R.U32 * tot.log()).all())
    assert abs(float(loss) - float(tot.log().mean())) <= 2 * R.U32 * float(loss)
    want = torch.empty(G, m, dtype=torch.float64, device="cuda")
    want[:, 1:] = (-z).exp() / tot[:, None] * 0.5 / G
    want[:, 0] = -want[:, 1:].sum(1)
    assert bool(((dlp.double().view(G, m) - want).abs() <= 2 * R.U32 * want.abs()).all())
    assert bool(((rewards.double() - 0.5 * lp.double()).abs() <= R.U32 * lp.double().abs()).all())
