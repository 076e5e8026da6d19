"""The LDS kernel with one activation row and a last stage wholly past the end
of K: the row is the whole buffer, so that stage starts behind it.

Tolerances are those of test_gpu_a4.py: sums here are exact in fp32, so
products are required to be equal; h has silu's error and one rounding."""

import pytest
import torch

from _gpu import DEV, say
from _launches import tiles
from test_gpu_a4_tiles import exact, f64, lo_scale, rand_mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


# blocks of K past a multiple of sixteen: 1, 2, 7 (the last stage is dead), 9
# and 15 (it is not); K with four, six and eight stages
@pytest.mark.parametrize("K", [544, 576, 736, 800, 992, 1056, 1248, 1632])
@pytest.mark.parametrize("M", [1, 2, 16])
def test_gemm(mm, M, K):
    say("gemm of few rows through LDS", M, K)
    gen = torch.Generator(device=DEV).manual_seed(M + K)
    lo = lo_scale(K)
    a, b = rand_mx(gen, (M,), K, lo, 127), rand_mx(gen, (50000,), K, lo, 127)
    assert tiles(lambda: mm.mxfp4_gemm(*a, *b)) == [("tiled", 2, 1, 0)]
    want = exact(f64(*a), f64(*b), lo, lo)
    assert torch.equal(mm.mxfp4_gemm(*a, *b).double(), want)
    assert torch.equal(mm.mxfp4_gemm(*a, *b, dtype=torch.bfloat16), want.float().to(torch.bfloat16))


def test_gate_up(mm):
    T, H, I, E, k = 1, 1056, 4096, 384, 8
    say("gate_up of one token through LDS", H, I, E, k)
    gen = torch.Generator(device=DEV).manual_seed(H)
    lo = lo_scale(H)
    x, w = rand_mx(gen, (T,), H, lo, 127), rand_mx(gen, (E, 2 * I), H, lo - 8, 119)
    ids = torch.randperm(E, device=DEV, generator=gen)[:k]
    pairs = torch.argsort(ids).int()
    offsets = torch.cat([torch.zeros(1, device=DEV), torch.bincount(ids, minlength=E).cumsum(0)]).int()
    args = (*x, pairs, offsets, k, *w)
    h = mm.moe_mxfp4_a4_gate_up_swiglu(*args)
    for call in (mm.moe_mxfp4_a4_gate_up_swiglu, mm.moe_mxfp4_a4_gate_up_swiglu_pack):
        assert tiles(lambda: call(*args)) == [("tiled", 4, 1, 0)]
    for row, e in enumerate(sorted(ids.tolist())):
        gu = exact(f64(*x), f64(w[0][e], w[1][e]), lo, lo - 8)[0]
        g, u = gu[:I], gu[I:]
        want = g * torch.sigmoid(g) * u
        tol = (2.0 ** -8 + 2.0 ** -21 * (2 + g.abs())) * want.abs() + 2.0 ** -126
        assert bool(((h[row].double() - want).abs() <= tol).all()), e
    pc, ps = mm.mxfp4_pack(h)
    hc, hs = mm.moe_mxfp4_a4_gate_up_swiglu_pack(*args)
    assert torch.equal(hc, pc) and torch.equal(hs, ps)
