"""The same contractions at the sizes that take each tile of the LDS kernel,
with K a multiple of 512 and not, against float64 on the GPU.

Every sum here is exact in fp32, whatever its order: the products are multiples
of 2^(2 (lo - 127) - 2), and the magnitudes of a sum stay below 2^24 of them
(asserted).  So products and down rows are required to be equal; h has the
tolerance of test_gpu_a4.py's test_gate_up (silu of an exact g, one product,
one rounding to bf16)."""

import pytest
import torch

from _gpu import DEV, say

pytestmark = pytest.mark.gpu

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def rand_mx(gen, shape, K, lo, hi):
    return [torch.randint(0, 256, (*shape, K // 2), dtype=torch.uint8, device=DEV, generator=gen),
            torch.randint(lo, hi + 1, (*shape, K // 32), dtype=torch.uint8, device=DEV, generator=gen)]


def f64(codes, scales):
    lut = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=DEV)
    v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def lo_scale(K):
    return 124 if K <= 1280 else 126


def exact(a, b, lo_a, lo_b):
    """a b^T, once it is shown to be exact in fp32."""
    mag = (a.abs() @ b.abs().T).max().item()
    assert mag < 2.0 ** 24 * 2.0 ** (lo_a + lo_b - 254 - 2)
    return a @ b.T


# tiles of 128 columns and 32, 64, 128 and 192 rows, and of 256 x 192
TILES = [(7, 13137, 2048), (7, 13137, 1632), (260, 2049, 2048), (260, 2049, 1184), (700, 2701, 1024),
         (700, 2702, 544), (1500, 2049, 512), (1500, 2051, 544), (7390, 771, 512), (4537, 1337, 544),
         (4537, 1337, 2048), (4540, 1340, 2080), (260, 2049, 2080), (4537, 2339, 2048), (4537, 2341, 2080),
         (8190, 3333, 2048), (8190, 3335, 2080)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_gemm_tiles(mm, M, N, K):
    say("gemm tiles", M, N, K)
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    lo = lo_scale(K)
    a, b = rand_mx(gen, (M,), K, lo, 127), rand_mx(gen, (N,), K, lo, 127)
    want = exact(f64(*a), f64(*b), lo, lo)
    out = torch.full((M + 2, N), -7.0, device=DEV)
    mm.mxfp4_gemm(*a, *b, out=out[1:M + 1])
    assert torch.equal(out[1:M + 1].double(), want)
    assert bool((out[0] == -7).all()) and bool((out[M + 1] == -7).all())
    out = torch.full((M + 2, N), -7.0, device=DEV, dtype=torch.bfloat16)
    mm.mxfp4_gemm(*a, *b, dtype=torch.bfloat16, out=out[1:M + 1])
    assert torch.equal(out[1:M + 1], want.float().to(torch.bfloat16))
    assert bool((out[0] == -7).all()) and bool((out[M + 1] == -7).all())


@pytest.mark.parametrize("M,N,K", [(7, 13137, 1632), (260, 2049, 1184), (260, 2049, 2048), (700, 2702, 544),
                                   (1500, 2051, 544), (4537, 1337, 544), (4537, 1337, 2048),
                                   (260, 2049, 2080), (4537, 2341, 2080), (8190, 3335, 2080)])
def test_gemm_tiles_nan_scales(mm, M, N, K):
    """A NaN block makes its own row (column) NaN and no other, first and last
    blocks of neighbouring rows among them."""
    say("gemm tiles nan", M, N, K)
    gen = torch.Generator(device=DEV).manual_seed(M + N)
    a, b = rand_mx(gen, (M,), K, 126, 127), rand_mx(gen, (N,), K, 126, 127)
    want = f64(*a) @ f64(*b).T
    rows, cols = [1, 4, M - 1], [0, 17, 18, N - 2]
    for i, r in enumerate(rows):
        a[1][r, (0, K // 32 - 1, 0)[i]] = 255
    for i, c in enumerate(cols):
        b[1][c, (K // 32 - 1, 0, K // 32 - 1, K // 64)[i]] = 255
    want[rows] = float("nan")
    want[:, cols] = float("nan")
    got = mm.mxfp4_gemm(*a, *b).double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("K", [512, 1024])
def test_gemm_tiles_unaligned_scales(mm, K):
    """Scale tensors that start at odd addresses, with rows of whole groups."""
    say("gemm tiles, scales at odd addresses", K)
    gen = torch.Generator(device=DEV).manual_seed(K)
    M, N = 1500, 2049
    a, b = rand_mx(gen, (M,), K, 126, 127), rand_mx(gen, (N,), K, 126, 127)
    want = exact(f64(*a), f64(*b), 126, 126)

    def shifted(s, by):
        room = torch.full((s.numel() + by,), 255, dtype=torch.uint8, device=DEV)
        room[by:] = s.flatten()
        return room[by:].view_as(s)

    got = mm.mxfp4_gemm(a[0], shifted(a[1], 3), b[0], shifted(b[1], 5))
    assert torch.equal(got.double(), want)


def routing(gen, T, E, k, skew):
    """sorted pair ids (garbage past the last segment), offsets, live rows:
    two pairs in a hundred dropped, the second expert left empty."""
    p = torch.arange(1, E + 1, device=DEV).double() ** -skew
    if E > k:
        p[1] = 0
    ids = torch.multinomial(p.expand(T, E), k, generator=gen)
    ids[torch.rand(T, k, device=DEV, generator=gen) < 0.02] = E
    flat = ids.flatten()
    order = torch.argsort(flat, stable=True).int()
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.cat([torch.zeros(1, device=DEV), counts.cumsum(0)]).int()
    n = int(offsets[-1])
    order[n:] = -1
    return order, offsets, n


# rows of a tile: 32, 64, 96; 32 and taller experts apart (two sizes); 64, 96;
# and more items than a workgroup lays out at a time
GATE_UP = [(1200, 1024, 544, 3, 1), (1200, 1056, 544, 3, 1), (1200, 1024, 1056, 3, 1),
           (1200, 1056, 1056, 3, 1), (1200, 1024, 1056, 3, 2), (1200, 1056, 1056, 3, 2),
           (200, 2048, 2080, 64, 2), (200, 2080, 2080, 64, 2), (700, 2048, 2080, 64, 4),
           (700, 2080, 2080, 64, 4), (1200, 1024, 2080, 9, 8), (1200, 1056, 2080, 9, 8),
           (1200, 2048, 2080, 8, 4), (1200, 2080, 2080, 8, 4), (2000, 1024, 1056, 1024, 4),
           (2000, 1056, 1056, 1024, 4)]


@pytest.mark.parametrize("T,H,I,E,k", GATE_UP)
def test_gate_up_tiles(mm, T, H, I, E, k):
    say("gate_up tiles", T, H, I, E, k)
    gen = torch.Generator(device=DEV).manual_seed(T + H + I + E + k)
    pairs, offsets, n = routing(gen, T, E, k, 1.0)
    lo = lo_scale(H)
    x, w = rand_mx(gen, (T,), H, lo, 127), rand_mx(gen, (E, 2 * I), H, lo - 8, 119)
    h = torch.full((T * k, I), -7.0, dtype=torch.bfloat16, device=DEV)
    mm.moe_mxfp4_a4_gate_up_swiglu(*x, pairs, offsets, k, *w, h=h)
    x64, off = f64(*x), offsets.tolist()
    for e in range(0, E, 1 if E < 100 else 13):
        if off[e] == off[e + 1]:
            continue
        rows = slice(off[e], off[e + 1])
        gu = exact(x64[pairs[rows].long() // k], f64(w[0][e], w[1][e]), lo, lo - 8)
        g, u = gu[:, :I], gu[:, I:]
        want = g * torch.sigmoid(g) * u
        tol = (2.0 ** -8 + 2.0 ** -21 * (2 + g.abs())) * want.abs() + 2.0 ** -126
        assert bool(((h[rows].double() - want).abs() <= tol).all()), e
    assert bool((h[n:] == -7).all()) and not bool((h[:n] == -7).all(1).any())
    hc = torch.full((T * k, I // 2), 0x5a, dtype=torch.uint8, device=DEV)
    hs = torch.full((T * k, I // 32), 0x5a, dtype=torch.uint8, device=DEV)
    mm.moe_mxfp4_a4_gate_up_swiglu_pack(*x, pairs, offsets, k, *w, h_codes=hc, h_scales=hs)
    pc, ps = mm.mxfp4_pack(h[:n].contiguous())
    assert torch.equal(hc[:n], pc) and torch.equal(hs[:n], ps)
    assert bool((hc[n:] == 0x5a).all()) and bool((hs[n:] == 0x5a).all())


DOWN = [(700, 1056, 512, 3, 1), (700, 1056, 1056, 3, 1), (1200, 1056, 512, 3, 2), (1200, 1056, 1056, 3, 2),
        (1200, 2080, 512, 3, 2), (1200, 2080, 1056, 3, 2), (1200, 2080, 2048, 9, 8), (1200, 2080, 2080, 17, 8),
        (300, 8192, 2048, 64, 4), (300, 8192, 2080, 64, 4), (700, 8192, 2048, 64, 4), (700, 8192, 2080, 64, 4),
        (2000, 2336, 512, 1024, 4), (2000, 2336, 1056, 1024, 4)]


@pytest.mark.parametrize("T,H,I,E,k", DOWN)
def test_down_tiles(mm, T, H, I, E, k):
    say("down tiles", T, H, I, E, k)
    gen = torch.Generator(device=DEV).manual_seed(T + H + I + E + k)
    _, offsets, n = routing(gen, T, E, k, 1.0)
    lo = lo_scale(I)
    h, w = rand_mx(gen, (T * k,), I, lo, 127), rand_mx(gen, (E, H), I, lo, 127)
    y = torch.full((T * k, H), -7.0, device=DEV)
    mm.moe_mxfp4_a4_down(*h, offsets, k, *w, y=y)
    off = offsets.tolist()
    for e in range(0, E, 1 if E < 100 else 13):
        rows = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            want = exact(f64(h[0][rows], h[1][rows]), f64(w[0][e], w[1][e]), lo, lo)
            assert torch.equal(y[rows].double(), want), e
    assert bool((y[n:] == -7).all()) and not bool((y[:n] == -7).all(1).any())
