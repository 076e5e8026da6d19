"""Weights of routing by scores within the errors of their own steps, path by path.

In units of 2^-24, relative: an exponential 2.5 (its instruction 2, its argument's
rounding 0.2); a quotient, a product and a sum's rounding 1 each; a sum of up to 32
taken scores 5 additions deep (4 where four tokens share a wave).
  sigmoid as it is      q / (1 + q): 2.5, 1 + q's rounding 1, the quotient 1 and the
                        factor 1: 5.5
  sigmoid renormalised  up / (1 + q): 2.5, 2.25 and 1; the same of the sum and its
                        5 additions, a quotient and the factor: 18.5
  softmax renormalised  2.5 twice, 5 additions, a quotient and the factor: 12
  softmax as it is      2.5 twice, the sum (fp64) rounded 1, a quotient and the factor:
                        8; four tokens a wave add up in fp32, 36 additions deep: 43
Scores stay within fp32's normal range here."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say
from oracle import scored

pytestmark = pytest.mark.gpu

UNITS = {(True, False): (5.5, 5.5), (True, True): (18.5, 18.5), (False, True): (12, 12), (False, False): (8, 43)}


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups", [(7, 384, 8, 8), (200, 1024, 32, 1), (300, 60, 12, 5), (4200, 384, 8, 8),
                                          (4200, 512, 8, 1), (4200, 24, 5, 2)])
def test_weights(mm, T, E, k, groups, sigmoid, norm):
    say("weights", T, E, k, sigmoid, norm)
    rng = np.random.default_rng([T, E, k, sigmoid, norm])
    logits = (rng.normal(0, 3, (T, E)) - 2 * rng.random((T, 1))).astype(np.float32)
    bias = (rng.integers(-60, 61, E) / 65536).astype(np.float32)
    some = rng.permutation(T)[:200]
    keep = max(1, groups // 2)
    for b in (bias, None):
        ids, w = mm.moe_route_scored(torch.from_numpy(logits).to(DEV), k, bias=None if b is None else torch.from_numpy(b).to(DEV),
                                     score="sigmoid" if sigmoid else "softmax", groups=groups, topk_groups=keep,
                                     renormalise=norm, scale=2.7)
        want, ww = scored.route(logits[some], k, b, sigmoid, groups, keep, 2, norm, float(np.float32(2.7)))
        assert np.array_equal(ids.cpu().numpy()[some], want)
        rel = np.abs(w.double().cpu().numpy()[some] - ww) / ww
        bound = UNITS[sigmoid, norm][T >= 4096]
        say("  worst %.2f units of %.1f" % (rel.max() * 2 ** 24, bound))
        assert rel.max() <= bound * 2.0 ** -24
