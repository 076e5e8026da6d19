"""Products of two MXFP4 factors whose sums lie below fp32's normal range.

Sums of multiples of 2^-149 are exact there, in any order, and required to be
equal.  Smaller products are rounded with each partial sum: K of those, each off
by at most 2^-149 (2^-23 of the magnitudes' sum above the normal range's end)."""

import pytest
import torch

from _gpu import DEV, say
from _launches import tiles
from test_gpu_a4_tiles import f64, rand_mx

pytestmark = pytest.mark.gpu

# the direct kernel's units, split and alone, and tiles of the other
SIZES = [(3, 40, 96, "direct"), (40, 300, 800, "direct"), (100, 2049, 1024, "direct"), (16, 50000, 544, "tiled"),
         (700, 2700, 992, "tiled"), (1500, 2701, 1024, "tiled")]


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


@pytest.mark.parametrize("M,N,K,kernel", SIZES)
@pytest.mark.parametrize("a_lo,b_lo", [(0, 127), (10, 97), (60, 47)])
def test_exact_down_to_the_last_bit(mm, M, N, K, kernel, a_lo, b_lo):
    """The smallest product, 2^(a_lo + b_lo - 256), is 2^-149 or more."""
    say("gemm of small values", M, N, K, a_lo, b_lo)
    gen = torch.Generator(device=DEV).manual_seed(M + N + K + a_lo)
    a, b = rand_mx(gen, (M,), K, a_lo, a_lo + 2), rand_mx(gen, (N,), K, b_lo, b_lo + 1)
    assert tiles(lambda: mm.mxfp4_gemm(*a, *b))[0][0] == kernel
    unit = 2.0 ** (a_lo + b_lo - 256)
    assert unit >= 2.0 ** -149 and (f64(*a).abs() @ f64(*b).abs().T).max().item() < 2.0 ** 24 * unit
    want = (f64(*a) @ f64(*b).T).cpu()
    assert 0 < want.abs().max().item() < 2.0 ** -112
    got = mm.mxfp4_gemm(*a, *b).cpu()
    assert torch.equal(got.double(), want)
    assert torch.equal(mm.mxfp4_gemm(*a, *b, dtype=torch.bfloat16).cpu(), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K,kernel", SIZES)
@pytest.mark.parametrize("a_lo,b_lo", [(0, 90), (0, 103), (0, 0), (50, 50)])
def test_products_below_the_spacing(mm, M, N, K, kernel, a_lo, b_lo):
    say("gemm of vanishing products", M, N, K, a_lo, b_lo)
    gen = torch.Generator(device=DEV).manual_seed(M + N + K + a_lo)
    a, b = rand_mx(gen, (M,), K, a_lo, a_lo + 12), rand_mx(gen, (N,), K, b_lo, b_lo + 12)
    assert tiles(lambda: mm.mxfp4_gemm(*a, *b))[0][0] == kernel
    x, y = f64(*a), f64(*b)
    want, mag = x @ y.T, x.abs() @ y.abs().T
    tol = K * (2.0 ** -149 + 2.0 ** -23 * mag)
    got = mm.mxfp4_gemm(*a, *b)
    assert bool(((got.double() - want).abs() <= tol).all())
    # one rounding to bf16, whose subnormals are spaced 2^-133
    half = mm.mxfp4_gemm(*a, *b, dtype=torch.bfloat16).double()
    assert bool(((half - got.double()).abs() <= 2.0 ** -8 * got.double().abs() + 2.0 ** -134).all())
