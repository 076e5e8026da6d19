"""dflash_verify_probs past 2^20 tokens, where a part of the vocabulary is more
than the draw takes at once.

Weights are multiples of 1/4 of at most 1, so every sum, and its product with a
24-bit uniform, is exact in float64 and the tokens are required to be equal;
test_rounded_away sets powers of two whose sums are not."""

import math

import numpy as np
import pytest
import torch

from _gpu import DEV, say
from oracle import verify_probs as ovp

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
VOCAB = [(1 << 20) + 1, (1 << 20) + 8, 3 * (1 << 20) + 5, 3 * (1 << 20) + 8]


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def part_length(V):
    """256 parts of whole groups of eight tokens; the draw takes 4096 at once."""
    return (math.ceil(V / 256) + 7) // 8 * 8


def call(mm, p, q, tokens, u, dtype):
    """One block; p [2, V], q [1, V] float64 of values that dtype holds."""
    up = lambda v: torch.from_numpy(v)[None].to(DEV).to(dtype)  # noqa: E731
    n, t = mm.dflash_verify_probs(up(p), up(q), torch.tensor([tokens], dtype=torch.int32, device=DEV),
                                  torch.tensor([u], dtype=torch.float32, device=DEV))
    return int(n), int(t)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("V", VOCAB)
def test_draws_in_every_round(mm, V, dtype):
    say("verify_probs long", V, dtype)
    rng = np.random.default_rng(V)
    p = rng.integers(0, 5, (2, V)) / 4.0
    q = rng.integers(0, 5, (1, V)) / 4.0
    span = part_length(V)
    assert span > 4096
    # tokens at the first, a middle and the last place of a part's rounds
    at = sorted({b + o for b in (0, 7 * span, (V - 1) // span * span, V // 2 // span * span)
                 for r in range(0, span, 4096) for o in (r, min(r + 2048, span - 1), min(r + 4095, span - 1))
                 if b + o < V})
    # the token to verify fails, passes (the draw is from row 1), or leaves no difference
    for case in ("residual", "whole", "equal"):
        qq, tokens, row = q, [-1], np.maximum(p[0] - q[0], 0)
        if case == "whole":
            d = int(np.flatnonzero((p[0] > 0) & (q[0] > 0))[0])
            tokens, row = [d], p[1]
        if case == "equal":
            qq, row = p[:1], p[0]
        c = np.cumsum(row)
        for t in at + [V - 1]:
            t = int(np.flatnonzero(row[t:])[0]) + t if row[t:].any() else int(np.flatnonzero(row)[-1])
            u = [0.0, float(np.float32((c[t] - row[t] / 2) / c[-1]))]
            want = ovp.verify_block(p, qq, tokens, u, 1)
            assert want == (int(case == "whole"), t)
            assert call(mm, p, qq, tokens, u, dtype) == want, (case, t)
        for u_draw, t in ((0.0, np.flatnonzero(row)[0]), (1.0 - 2.0 ** -24, None)):
            want = ovp.verify_block(p, qq, tokens, [0.0, u_draw], 1)
            assert t is None or want[1] == t
            assert call(mm, p, qq, tokens, [0.0, u_draw], dtype) == want, (case, u_draw)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("V", VOCAB)
def test_few_tokens(mm, V, dtype):
    """One token of a part, in any of its rounds; none at all."""
    say("verify_probs long, few tokens", V, dtype)
    span = part_length(V)
    q = np.zeros((1, V))
    for t in (0, span - 1, 5 * span + 4095, 5 * span + 4096, 6 * span - 1, V - 1):
        p = np.zeros((2, V))
        p[0, t] = 0.25
        for u in (0.0, 0.5, 1.0 - 2.0 ** -24):
            assert call(mm, p, q, [-1], [0.0, u], dtype) == (0, t)
    assert call(mm, np.zeros((2, V)), q, [-1], [0.0, 0.5], dtype) == (0, -1)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_rounded_away(mm, dtype):
    """Weights 1, 2^-54, 2^-53, 1 and u = 1/2: the goal, 1 + 1.5 2^-54, lies in
    the weight of 2^-53.  In float64 the part of the small ones ends at
    1 + 2^-52, past the rounded goal of 1, but within it every running sum
    rounds to 1: no token is hit, and the last with weight is taken, of an
    earlier round than the part's last."""
    V = 3 * (1 << 20) + 5
    say("verify_probs long, rounded away", dtype)
    span = part_length(V)
    first, second = span + 11, span + 4096 + 17
    p = np.zeros((2, V))
    p[0, [0, first, second, V - 1]] = [1.0, 2.0 ** -54, 2.0 ** -53, 1.0]
    assert call(mm, p, np.zeros((1, V)), [-1], [0.0, 0.5], dtype) == (0, second)
