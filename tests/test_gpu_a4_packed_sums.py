"""gate/up with h in MXFP4 where the sums are rounded: a wide range of scales, at
sizes where the packed form takes another kernel, or order of summation, than
the bf16 one.

Both forms are held to the definition in float64.  A sum of K exact products is
off by at most K 2^-23 of their magnitudes' sum; |silu'| is below 1.1 and silu
as computed off by 2^-21 (2 + |g|) of itself; h is rounded to bf16, 2^-8.  That
gives each h an interval.  Conversion is monotonic, so a block's scale lies
between those of its intervals' ends and each value, under the scale that was
written, between its interval's ends rounded to E2M1."""

import pytest
import torch

from _gpu import DEV, say
from _launches import tiles
from test_gpu_a4_tiles import f64, rand_mx, routing

pytestmark = pytest.mark.gpu

# the last two: the same order in both forms
SIZES = [(200, 2080, 2080, 64, 2), (60, 2048, 2048, 8, 2), (100, 512, 1024, 16, 2), (1007, 480, 96, 85, 6),
         (12, 4096, 512, 8, 2), (900, 1056, 1056, 9, 4)]


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def intervals(x, w, K, I):
    """(low, high) [rows, I] of h before its rounding to bf16."""
    gu, mag = x @ w.T, x.abs() @ w.abs().T
    g, u = gu[:, :I], gu[:, I:]
    dg, du = K * 2.0 ** -23 * mag[:, :I], K * 2.0 ** -23 * mag[:, I:]
    s = g * torch.sigmoid(g)
    h = s * u
    off = 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + 2.0 ** -21 * (2 + g.abs() + dg) * h.abs() + 2.0 ** -126
    return h - off, h + off


def rounded(v):
    """v (scaled) to the nearest E2M1 value, saturating."""
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], dtype=torch.float64, device=DEV)
    return values[torch.bucketize(v.abs(), mids)] * v.sign()


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_both_forms(mm, T, H, I, E, k):
    say("packed gate_up, rounded sums", T, H, I, E, k)
    gen = torch.Generator(device=DEV).manual_seed(T + H + I)
    pairs, offsets, n = routing(gen, T, E, k, 1.0)
    x, w = rand_mx(gen, (T,), H, 105, 127), rand_mx(gen, (E, 2 * I), H, 98, 120)
    args = (*x, pairs, offsets, k, *w)
    say("  bf16", tiles(lambda: mm.moe_mxfp4_a4_gate_up_swiglu(*args)),
        "packed", tiles(lambda: mm.moe_mxfp4_a4_gate_up_swiglu_pack(*args)))
    h = mm.moe_mxfp4_a4_gate_up_swiglu(*args)
    hc, hs = mm.moe_mxfp4_a4_gate_up_swiglu_pack(*args)
    x64, off = f64(*x), offsets.tolist()
    certain = total = 0
    for e in range(0, E, max(1, E // 16)):
        rows = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        lo, hi = intervals(x64[pairs[rows].long() // k], f64(w[0][e], w[1][e]), H, I)
        lo, hi = lo - 2.0 ** -8 * lo.abs() - 2.0 ** -134, hi + 2.0 ** -8 * hi.abs() + 2.0 ** -134
        got = h[rows].double()
        assert bool(((got >= lo) & (got <= hi)).all()), e
        # scales: floor(log2 of the largest magnitude) - 2, biased
        blocks = lambda t: t.view(t.shape[0], I // 32, 32)  # noqa: E731
        least = torch.where((lo <= 0) & (hi >= 0), 0.0, torch.minimum(lo.abs(), hi.abs()))
        most = torch.maximum(lo.abs(), hi.abs())
        byte = lambda m: (torch.frexp(m).exponent - 1 - 2 + 127).clamp(0, 254)  # noqa: E731
        s_lo, s_hi = byte(blocks(least).amax(2).clamp_min(2.0 ** -140)), byte(blocks(most).amax(2))
        s = hs[rows].long()
        assert bool(((s >= s_lo) & (s <= s_hi)).all()), e
        scale = torch.exp2(s.double() - 127).repeat_interleave(32, 1)
        value = f64(hc[rows], hs[rows]) / scale
        a, b = rounded(lo / scale), rounded(hi / scale)
        assert bool(((value >= a) & (value <= b)).all()), e
        certain += int((a == b).sum())
        total += a.numel()
    say("  codes that the bounds leave one value: %d of %d" % (certain, total))
