"""The contractions through the LDS kernel at every length of K past a multiple
of 512 (the last stages part full or empty, scale rows at every distance from
the 16 bytes they are loaded by), for each tile.  Every test asserts which
kernels its call launches.

Tolerances are those of test_gpu_a4_tiles.py: sums are exact in fp32 (shown
each time), so products and down rows are required to be equal; h has silu's
error and one rounding."""

import pytest
import torch

from _gpu import DEV, say
from _launches import tiles
from test_gpu_a4_tiles import exact, f64, lo_scale, rand_mx, routing

pytestmark = pytest.mark.gpu

LENGTHS, LONGER = range(544, 1025, 32), range(800, 1281, 32)


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


# T, I, E, k, the row subtiles of the launches (one tile height, or the experts
# that outgrow the tile in a launch before; 192 rows are 160 where K is not
# whole) and the lengths that take them: below 800 only experts of more than 64
# rows as a rule
GATE_UP = [(500, 544, 16, 1, (1,), LONGER), (300, 288, 16, 8, (2,), LENGTHS), (4000, 288, 16, 1, (2,), LENGTHS),
           (500, 2080, 8, 1, (3,), LENGTHS), (200, 1056, 384, 8, (3, 1), LONGER),
           (900, 2080, 128, 4, (6, 2), LONGER), (900, 2080, 64, 8, (6, 3), LENGTHS)]


@pytest.mark.parametrize("T,I,E,k,ms,lengths", GATE_UP)
def test_gate_up(mm, T, I, E, k, ms, lengths):
    for H in lengths:
        say("gate_up lengths", T, H, I, E, k)
        gen = torch.Generator(device=DEV).manual_seed(T + H + I + E + k)
        pairs, offsets, n = routing(gen, T, E, k, 1.0)
        lo = lo_scale(H)
        x, w = rand_mx(gen, (T,), H, lo, 127), rand_mx(gen, (E, 2 * I), H, lo - 8, 119)
        args = (*x, pairs, offsets, k, *w)
        whole = int(H % 512 == 0)
        launches = [("tiled", 4, 5 if m == 6 and not whole else m, whole) for m in ms]
        for call in (mm.moe_mxfp4_a4_gate_up_swiglu, mm.moe_mxfp4_a4_gate_up_swiglu_pack):
            assert tiles(lambda: call(*args)) == launches, H
        h = torch.full((T * k, I), -7.0, dtype=torch.bfloat16, device=DEV)
        mm.moe_mxfp4_a4_gate_up_swiglu(*args, h=h)
        x64, off = f64(*x), offsets.tolist()
        for e in range(0, E, max(1, E // 16)):
            rows = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            gu = exact(x64[pairs[rows].long() // k], f64(w[0][e], w[1][e]), lo, lo - 8)
            g, u = gu[:, :I], gu[:, I:]
            want = g * torch.sigmoid(g) * u
            tol = (2.0 ** -8 + 2.0 ** -21 * (2 + g.abs())) * want.abs() + 2.0 ** -126
            assert bool(((h[rows].double() - want).abs() <= tol).all()), (H, e)
        assert bool((h[n:] == -7).all()) and not bool((h[:n] == -7).all(1).any())
        hc = torch.full((T * k, I // 2), 0x5a, dtype=torch.uint8, device=DEV)
        hs = torch.full((T * k, I // 32), 0x5a, dtype=torch.uint8, device=DEV)
        mm.moe_mxfp4_a4_gate_up_swiglu_pack(*args, h_codes=hc, h_scales=hs)
        pc, ps = mm.mxfp4_pack(h[:n].contiguous())
        assert torch.equal(hc[:n], pc) and torch.equal(hs[:n], ps)
        assert bool((hc[n:] == 0x5a).all()) and bool((hs[n:] == 0x5a).all())


@pytest.mark.parametrize("T,I,E,k", [(8, 2048, 64, 8), (500, 544, 16, 1)])
def test_gate_up_short_and_few_rows(mm, T, I, E, k):
    """Below K = 800 experts of few rows stay on the direct kernel."""
    for H in (544, 640, 768):
        gen = torch.Generator(device=DEV).manual_seed(H)
        pairs, offsets, _ = routing(gen, T, E, k, 1.0)
        args = (*rand_mx(gen, (T,), H, 124, 127), pairs, offsets, k, *rand_mx(gen, (E, 2 * I), H, 116, 119))
        for call in (mm.moe_mxfp4_a4_gate_up_swiglu, mm.moe_mxfp4_a4_gate_up_swiglu_pack):
            assert [t[0] for t in tiles(lambda: call(*args))] == ["direct"], H
