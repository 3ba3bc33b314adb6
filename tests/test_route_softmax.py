"""Softmax routing with experts that a bias of -inf takes out of the choice."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LOWEST = -3.4028234663852886e38


# Experts per lane on both sides of 2, 4, 8 and 16, one and several groups.
SHAPES = [(16, 8, 1, 1), (64, 6, 8, 3), (128, 8, 1, 1), (130, 6, 2, 1), (256, 8, 1, 1),
          (300, 8, 1, 1), (512, 8, 1, 1), (576, 8, 1, 1), (896, 16, 8, 4), (1024, 16, 1, 1),
          (1088, 9, 1, 1), (2048, 16, 1, 1), (1056, 12, 4, 3)]


@pytest.mark.parametrize("E,K,G,KG", SHAPES)
def test_bias_of_minus_infinity_keeps_its_share_of_the_softmax(E, K, G, KG):
    """The weights are softmax values over every expert that its logit does not mask; a bias of
    -inf takes an expert out of the choice only.  Expected values by torch.softmax in 64 bits."""
    import mxfp8_mxfp4_experts_amd as m
    T, per = 24, E // G
    g = torch.Generator().manual_seed(E + K)
    l = 1.5 * torch.randn(T, E, generator=g)
    out = torch.rand(E, generator=g) < 0.25            # by their biases
    out[0], out[1] = True, False
    l[:, 0] = 3.0                                      # one of them with a large share
    hidden = torch.rand(T, E, generator=g) < 0.1       # by their logits
    l = torch.where(hidden, torch.where(torch.rand(T, E, generator=g) < 0.5, -math.inf, LOWEST), l)
    l[5, ~out] = -math.inf                             # a token that only they could take
    bias = torch.where(out, -math.inf, 0.0)
    idx, w = m.moe_route_groups(l.cuda(), bias.cuda(), K, n_group=G, topk_group=KG,
                                score=m.SCORE_SOFTMAX, group_score=m.GROUP_MAX, renormalise=False)
    s = torch.softmax(torch.where(l <= LOWEST, -math.inf, l).double(), 1)
    key = torch.where(out | (l <= LOWEST), -math.inf, s.float().double())
    best = key.view(T, G, per).amax(2)
    kept = torch.zeros(T, G, dtype=torch.bool)
    kept.scatter_(1, best.sort(dim=1, descending=True, stable=True)[1][:, :KG], True)
    key = torch.where(kept.repeat_interleave(per, 1), key, -math.inf)
    val, want = key.sort(dim=1, descending=True, stable=True)
    none = val[:, :K] == -math.inf
    want = torch.where(none, -1, want[:, :K])
    assert (want[5] == -1).all() and not none[0, 0]
    assert np.array_equal(idx.cpu().numpy(), want.numpy())
    sw = torch.where(none, 0.0, s.gather(1, want.clamp_min(0)))
    # a score is rounded to float once (2^-24), times a scaling of 1; the doubles' own errors are
    # far below the other half
    assert ((w.cpu().double() - sw).abs() <= 2.0 ** -23 * sw).all()
