"""Two experts whose values c = s + b differ by a few units in fp32's last place of
their scores' difference: fp32 settles their order where its error cannot turn it,
and fp64 the rest, so the better one in 64 bits comes first.

Each pair has the biases 0 and beta, a logit l of the second and for the first one
of the numbers next to the h whose score is s(l) + beta.  A step of h changes c
by about 2^-23 of s(h) - s(l); distances h - l lie on both sides of 1/2, where the
kernel changes from a series to an exponential."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v.astype(np.float64)))


def pairs(rng, n, beta):
    """float32 h, l [n]: sigmoid(h) next to sigmoid(l) + beta."""
    lo = (rng.normal(0, 2, n)).astype(np.float32)
    want = sigmoid(lo) + beta
    lo, want = lo[want < 0.999], want[want < 0.999]
    h = np.log(want / (1.0 - want)).astype(np.float32)
    steps = rng.integers(-24, 25, len(h))
    up = np.nextafter(h, np.float32(np.inf)) - h
    return (h + steps.astype(np.float32) * up).astype(np.float32), lo


BETAS = [2.0 ** -10, 0.01, 0.03, 0.06, 0.09, 0.11, 0.12, 0.125, 0.14, 0.17, 0.2, 0.25, 0.3, 0.4, 0.6]


@pytest.mark.parametrize("E", [2, 8], ids=["token", "rows"])
def test_sigmoid(mm, E):
    """One token a wave (two experts), and four (eight, six of them far below)."""
    rng = np.random.default_rng(E)
    wrong = total = near = 0
    for beta in BETAS:
        beta = np.float32(beta)
        h, lo = pairs(rng, 400000, float(beta))
        logits = np.full((len(h), E), -60.0, np.float32)
        logits[:, 0], logits[:, 1] = h, lo
        bias = np.zeros(E, np.float32)
        bias[1] = beta
        x = sigmoid(h) - (sigmoid(lo) + float(beta))
        ids, _ = mm.moe_route_scored(torch.from_numpy(logits).to(DEV), 1, bias=torch.from_numpy(bias).to(DEV))
        got = ids.cpu().numpy()[:, 0]
        sure = np.abs(x) > 2.0 ** -50                     # else fp64 rounds either way
        bad = (got != np.where(x >= 0, 0, 1)) & sure
        rel = np.abs(x) / np.abs(sigmoid(h) - sigmoid(lo))
        wrong, total, near = wrong + int(bad.sum()), total + len(h), near + int((rel < 2.0 ** -19).sum())
        say("  beta %-10g pairs %d, within 2^-20 %d, 2^-19 %d, wrong %d%s" % (
            beta, len(h), (rel < 2.0 ** -20).sum(), (rel < 2.0 ** -19).sum(), bad.sum(),
            ", the furthest 2^%.2f" % np.log2(rel[bad].max()) if bad.any() else ""))
    assert near > total // 20
    assert wrong == 0
