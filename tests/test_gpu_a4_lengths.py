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


# T, H, E, k and the row subtiles of the launches
DOWN = [(200, 2080, 3, 1, (1,)), (500, 288, 8, 8, (2,)), (500, 544, 32, 8, (3,)),
        (200, 2080, 384, 8, (3, 1)), (900, 4128, 128, 4, (6, 2)), (900, 4128, 64, 8, (6, 3))]


@pytest.mark.parametrize("T,H,E,k,ms", DOWN)
def test_down(mm, T, H, E, k, ms):
    for I in LENGTHS:
        say("down lengths", T, H, I, E, k)
        gen = torch.Generator(device=DEV).manual_seed(T + H + I + E + k)
        _, offsets, n = routing(gen, T, E, k, 1.0)
        lo = lo_scale(I)
        h, w = rand_mx(gen, (T * k,), I, lo, 127), rand_mx(gen, (E, H), I, lo, 127)
        assert tiles(lambda: mm.moe_mxfp4_a4_down(*h, offsets, k, *w)) == \
            [("tiled", 4, m, int(I % 512 == 0)) for m in ms], I
        y = torch.full((T * k, H), -7.0, device=DEV)
        mm.moe_mxfp4_a4_down(*h, offsets, k, *w, y=y)
        off = offsets.tolist()
        for e in range(0, E, max(1, E // 16)):
            rows = slice(off[e], off[e + 1])
            if off[e] < off[e + 1]:
                want = exact(f64(h[0][rows], h[1][rows]), f64(w[0][e], w[1][e]), lo, lo)
                assert torch.equal(y[rows].double(), want), (I, e)
        assert bool((y[n:] == -7).all()) and not bool((y[:n] == -7).all(1).any())


GEMM = [(16, 50000, (2, 1), LENGTHS), (700, 2700, (2, 2), LENGTHS), (2100, 1001, (2, 4), LENGTHS),
        (1500, 2701, (2, 6), LENGTHS), (4537, 2051, (4, 6), range(2048, 2529, 32))]


@pytest.mark.parametrize("M,N,tile,lengths", GEMM)
def test_gemm(mm, M, N, tile, lengths):
    for K in lengths:
        say("gemm lengths", M, N, K)
        gen = torch.Generator(device=DEV).manual_seed(M + N + K)
        lo = lo_scale(K)
        a, b = rand_mx(gen, (M,), K, lo, 127), rand_mx(gen, (N,), K, lo, 127)
        want = exact(f64(*a), f64(*b), lo, lo)
        for dtype in (torch.float32, torch.bfloat16):
            assert tiles(lambda: mm.mxfp4_gemm(*a, *b, dtype=dtype)) == [("tiled", *tile, int(K % 512 == 0))], K
            out = torch.full((M + 2, N), -7.0, device=DEV, dtype=dtype)
            mm.mxfp4_gemm(*a, *b, dtype=dtype, out=out[1:M + 1])
            assert torch.equal(out[1:M + 1], want.float().to(dtype)), K
            assert bool((out[0] == -7).all()) and bool((out[M + 1] == -7).all())


# sizes of the direct kernel's units and of the tiles above
SPECIAL = [(40, 65, "direct"), (60, 1301, "direct"), (40, 2049, "direct"), (100, 2049, "direct"),
           (16, 50000, "tiled"), (700, 2700, "tiled"), (1500, 2701, "tiled")]


@pytest.mark.parametrize("M,N,kernel", SPECIAL)
def test_gemm_nan_scales(mm, M, N, kernel):
    """A NaN block makes its row (column) NaN and no other, whatever the block
    and its neighbours' last and first ones."""
    for K in LENGTHS:
        say("gemm lengths, nan", M, N, K)
        gen = torch.Generator(device=DEV).manual_seed(M + N + K)
        a, b = rand_mx(gen, (M,), K, 124, 127), rand_mx(gen, (N,), K, 124, 127)
        assert tiles(lambda: mm.mxfp4_gemm(*a, *b))[0][0] == kernel, K
        want = exact(f64(*a), f64(*b), 124, 124)
        last = K // 32 - 1
        rows, blocks = [1, 2, 4, 9, M - 1], [0, last, 0, 16, last - 1]
        cols, col_blocks = [0, 17, 18, N // 2, N - 2], [last, 0, last, 15, last // 2]
        a[1][rows, blocks] = 255
        b[1][cols, col_blocks] = 255
        want[rows] = float("nan")
        want[:, cols] = float("nan")
        got = mm.mxfp4_gemm(*a, *b).double()
        assert torch.equal(got.isnan(), want.isnan()), K
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)), K


@pytest.mark.parametrize("M,N,kernel", SPECIAL)
def test_gemm_zeros_under_the_largest_scales(mm, M, N, kernel):
    """A zero code times 2^127 times a value under 2^127 is zero, in the blocks
    of K and in the empty ones past its end."""
    for K in LENGTHS:
        say("gemm lengths, zeros under 2^127", M, N, K)
        gen = torch.Generator(device=DEV).manual_seed(M + N + K)
        a, b = rand_mx(gen, (M,), K, 124, 127), rand_mx(gen, (N,), K, 124, 127)
        assert tiles(lambda: mm.mxfp4_gemm(*a, *b))[0][0] == kernel, K
        b[1][1::3] = 254                             # a third of the columns: 2^127 but in the live blocks
        for m in (0, 3, M - 1):                      # these rows: zeros but for one block
            live = (m + K // 32) % (K // 32)
            for t, fill in ((a[0], 0), (a[1], 254)):
                keep = t[m].view(K // 32, -1)[live].clone()
                t[m] = fill
                t[m].view(K // 32, -1)[live] = keep
            b[1][1::3, live] = 125
        want = f64(*a)[[0, 3, M - 1]] @ f64(*b).T
        got = mm.mxfp4_gemm(*a, *b)[[0, 3, M - 1]].double()
        assert torch.equal(got, want), K
