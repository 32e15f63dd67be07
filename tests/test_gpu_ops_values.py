"""Infinities and NaN in the losses on log-probabilities: what counts passes them on, what does not count never does."""
import math

import pytest
import torch

import catalogue_cross_entropy_amd as rece

pytestmark = pytest.mark.gpu
KINDS = ["sigmoid", "ipo", "hinge", "softmax"]


def _pairs(G, per, members=2):
    """Offsets of G groups of `members` sequences of `per` tokens."""
    offs = (torch.arange(G * members + 1) * per).to(torch.int32).cuda()
    return offs, (torch.arange(G + 1) * members).to(torch.int32).cuda()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,per", [(5, 3), (5, 100), (9000, 1), (9000, 6)])
@pytest.mark.parametrize("which", [0, 1])
def test_preference_nan_is_not_swallowed(kind, G, per, which):
    """A NaN in a token that counts makes its group's loss NaN, and the mean, and its group's gradients; no other's."""
    offs, goffs = _pairs(G, per)
    n = G * 2 * per
    lp = -torch.rand(n, generator=torch.Generator().manual_seed(G))
    lp[(2 * 3 + which) * per] = float("nan")   # a token of group 3
    print(f"[gpu] preference NaN {kind} G={G} per={per}", flush=True)
    loss, pg, rewards, dlp = rece.PreferenceLoss(n, 2 * G, G, kind=kind).forward(lp.cuda(), None, offs, goffs)
    group = torch.arange(G) == 3
    assert math.isnan(float(loss)) and torch.equal(pg.isnan().cpu(), group)
    assert torch.equal(dlp.isnan().cpu().view(G, -1), group[:, None].expand(G, 2 * per))
    assert torch.equal(rewards.isnan().cpu(), torch.arange(2 * G) == 6 + which)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [300, 20000])
@pytest.mark.parametrize("up", [float("inf"), float("nan")])
def test_policy_tokens_that_do_not_count_get_zero_whatever_dloss_is(n, up, dtype):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    lp = (-torch.rand(n, generator=torch.Generator().manual_seed(n))).to(dt).cuda()
    mask = torch.arange(n, device="cuda") % 3 > 0
    offs = torch.tensor([5, n // 2, n - 4], dtype=torch.int32, device="cuda")
    op = rece.PolicyLoss(n, 2, entropy_coef=0.1, dtype=dtype)
    _, _, dlp, dH = op.forward(lp, lp, torch.ones(2, device="cuda"), offs, entropy=-lp, mask=mask,
                               dloss=torch.tensor([up], device="cuda"))
    at = torch.arange(n, device="cuda")
    on = mask & (at >= 5) & (at < n - 4)
    for v in (dlp, dH):
        assert not bool(v[~on].any()) and not bool(v[on].isfinite().any())


@pytest.mark.parametrize("G,per", [(4, 1), (4, 80), (9000, 1), (9000, 5)])
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_preference_of_an_impossible_rejected_sequence(kind, G, per):
    """A rejected sequence of log-probability minus infinity: that group's loss is 0 and moves nothing."""
    offs, goffs = _pairs(G, per)
    n = G * 2 * per
    lp = -torch.rand(n, generator=torch.Generator().manual_seed(3))
    lp[(2 * 2 + 1) * per] = float("-inf")
    loss, pg, _, dlp = rece.PreferenceLoss(n, 2 * G, G, kind=kind).forward(lp.cuda(), None, offs, goffs)
    assert float(pg[2]) == 0.0 and bool(pg.isfinite().all()) and math.isfinite(float(loss))
    grads = dlp.view(G, -1)
    assert not bool(grads[2].any()) and bool(grads[:2].all()) and bool(grads.isfinite().all())


@pytest.mark.parametrize("G,per", [(4, 1), (4, 80), (9000, 1), (9000, 5)])
@pytest.mark.parametrize("kind", ["sigmoid", "softmax", "hinge"])
@pytest.mark.parametrize("members", [2, 3])
def test_preference_of_an_impossible_preferred_sequence(kind, G, per, members):
    """A preferred sequence of log-probability minus infinity: an infinite loss, with the slope it has there."""
    offs, goffs = _pairs(G, per, members)
    n = G * members * per
    lp = -torch.rand(n, generator=torch.Generator().manual_seed(4))
    lp[2 * members * per] = float("-inf")
    op = rece.PreferenceLoss(n, members * G, G, beta=0.5, kind=kind)
    loss, pg, _, dlp = op.forward(lp.cuda(), None, offs, goffs)
    assert float(pg[2]) == math.inf and float(loss) == math.inf and bool(pg.isfinite().cpu()[torch.arange(G) != 2].all())
    got = dlp.view(G, members, per)[2].cpu().double()
    want = torch.full((members, per), 0.5 / G / (members - 1), dtype=torch.float64)
    want[0] = -0.5 / G
    assert bool(((got - want).abs() <= 2.0 ** -23 * want.abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("s,C", [(3, 20), (5, 700), (300, 45)])
def test_logprob_at_the_ends_of_its_temperatures(s, C, dtype):
    """2^64: all items alike, whatever the logits (below 2^-50 here).  2^-20: the best item alone (others are 2^10 below)."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator().manual_seed(C)
    X = torch.ones(s, 32)
    Y = torch.zeros(C, 32)
    Y[:, 0] = torch.randperm(C, generator=g) / 1024.0 - 0.3   # all different, exact in bf16 up to 256 of them
    Y = Y.to(dt)
    best = int(Y[:, 0].float().argmax())
    ids = torch.randint(0, C, (s,), generator=g).to(torch.int32)
    ids[0] = best
    args = (X.to(dt).cuda(), Y.cuda(), ids.cuda())
    for T in (2.0 ** 64, 2.0 ** -20):
        op = rece.LogProb(s, C, 32, dtype=dtype, temperature=T, entropy=True)
        logp, ent, ws = op.forward(*args)
        dX, dY = op.backward(*args, ws, torch.full((s,), T, device="cuda"))
        assert bool(dX.isfinite().all()) and bool(dY.isfinite().all())
        if T > 1:
            want = -float(torch.tensor(float(C), dtype=torch.float64).log())
            assert bool(((logp.cpu().double() - want).abs() <= 16 * 2.0 ** -24 * abs(want)).all())
            assert bool(((ent.cpu().double() + want).abs() <= 16 * 2.0 ** -24 * abs(want)).all())
        elif int((Y[:, 0] == Y[best, 0]).sum()) == 1:
            hit = ids == best
            assert bool((logp.cpu()[hit] == 0).all()) and bool((logp.cpu()[~hit] < -2.0 ** 9).all())
