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
