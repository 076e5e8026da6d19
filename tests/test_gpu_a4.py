"""GPU parity of the products of two MXFP4 factors with the float64 oracle.

Tolerances.  Products are exact, so a sum of K of them in fp32 is off by at
most K roundings (or truncations) of 2^-23 of the magnitudes' sum.  Inputs
with a narrow range of scales do better: every partial sum is a multiple of
the smallest product and below 2^24 of them, so the result is exact whatever
the order, and is required to be.  h adds silu(g) u: the exponential of an
fp32 argument is off by 2^-22 (1 + |g|) relative, the division and the
product by another 2^-22, then one rounding to bf16, 2^-8."""

import numpy as np
import pytest
import torch

from _gpu import DEV, host_bits, say
from oracle import a4 as oa4
from oracle import mx as omx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def mx(rng, shape, K, lo=124, hi=127):
    return (rng.integers(0, 256, (*shape, K // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (*shape, K // 32), dtype=np.uint8))


def up(pair):
    return [torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in pair]


def sum_bound(K, mag):
    return K * 2.0 ** -23 * mag


GEMM = [(1, 1, 32), (1, 16, 64), (2, 3, 96), (3, 40, 128), (16, 16, 256), (17, 33, 160),
        (8, 300, 1024), (33, 64, 288), (64, 256, 512), (65, 257, 544), (130, 100, 2080),
        (257, 513, 768), (300, 600, 1280), (512, 256, 256), (40, 1030, 2048), (129, 260, 4096)]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm_exact_sums(mm, M, N, K):
    say("gemm exact", M, N, K)
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    # products are multiples of 2^-8 (scales 2^-3 .. 2^0 on both sides) of at
    # most 36; 2080 of them stay below 2^24 2^-8; longer sums use fewer scales
    lo = 124 if K <= 1280 else 126
    a, b = mx(rng, (M,), K, lo), mx(rng, (N,), K, lo)
    want, mag = oa4.gemm(*a, *b)
    assert mag.max() < 2.0 ** 24 * 2.0 ** (2 * (lo - 127) - 2)
    got = mm.mxfp4_gemm(*up(a), *up(b)).cpu().numpy()
    assert np.array_equal(got.astype(np.float64), want)
    got = mm.mxfp4_gemm(*up(a), *up(b), dtype=torch.bfloat16)
    assert np.array_equal(host_bits(got), omx.to_bf16_bits(want))


@pytest.mark.parametrize("M,N,K", [(5, 70, 2080), (48, 48, 6144), (200, 300, 1024), (260, 256, 4096)])
def test_gemm_wide_scales(mm, M, N, K):
    say("gemm wide", M, N, K)
    rng = np.random.default_rng(K + N)
    a, b = mx(rng, (M,), K, 100, 150), mx(rng, (N,), K, 90, 140)
    want, mag = oa4.gemm(*a, *b)
    got = mm.mxfp4_gemm(*up(a), *up(b)).cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= sum_bound(K, mag))
    got = omx.bf16_bits_to_f64(host_bits(mm.mxfp4_gemm(*up(a), *up(b), dtype=torch.bfloat16)))
    assert np.all(np.abs(got - want) <= sum_bound(K, mag) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want))


@pytest.mark.parametrize("M,N,K", [(4, 20, 96), (20, 40, 512), (140, 260, 800), (260, 300, 1024)])
def test_gemm_extreme_scale_bytes(mm, M, N, K):
    """Byte 0 is 2^-127, byte 255 NaN: only that row (column) is NaN."""
    say("gemm bytes", M, N, K)
    rng = np.random.default_rng(N)
    a, b = mx(rng, (M,), K), mx(rng, (N,), K)
    a[1][0, :] = 0                                   # row 0: 2^-127 throughout
    b[1][1, :] = 254                                 # column 1: 2^127 throughout
    a[1][2, K // 32 - 1] = 255                       # row 2: its last block is NaN
    b[1][3, 0] = 255
    b[1][N - 1, K // 64] = 255
    want, mag = oa4.gemm(*a, *b)
    got = mm.mxfp4_gemm(*up(a), *up(b)).cpu().numpy().astype(np.float64)
    nan = np.zeros((M, N), bool)
    nan[2], nan[:, 3], nan[:, N - 1] = True, True, True
    # where the products' magnitudes sum to 2^128 and more (2^127 times up to
    # 36 K 2^-3 in column 1) fp32 may overflow on the way, in any order, and
    # opposite infinities meet: those entries are Inf or NaN
    fits = nan | (mag < 2.0 ** 128)
    assert np.all(fits[:, [0, 2]]) and np.all(fits[0])
    assert np.array_equal(np.isnan(got)[fits], nan[fits])
    assert np.array_equal(np.isnan(want), nan)
    ok = ~nan & fits
    ok[0, :] = False                                 # below fp32's normal range but for column 1
    assert np.array_equal(got[ok], want[ok])
    assert got[0, 1] == want[0, 1]                   # 2^-127 2^127: exact
    assert np.all(np.abs(got[0][~nan[0]] - want[0][~nan[0]]) <= 2.0 ** -100)


def test_gemm_empty_and_views(mm):
    say("gemm empty and views")
    rng = np.random.default_rng(5)
    a, b = up(mx(rng, (40,), 32)), up(mx(rng, (30,), 32))
    assert mm.mxfp4_gemm(a[0][:0], a[1][:0], *b).shape == (0, 30)
    assert mm.mxfp4_gemm(*a, b[0][:0], b[1][:0]).shape == (40, 0)
    whole = mm.mxfp4_gemm(*a, *b)
    # views: codes rows stay 16-byte aligned, scale rows and outputs do not
    out = torch.full((41, 29), -7.0, device=DEV)
    mm.mxfp4_gemm(a[0][3:], a[1][3:], b[0][1:], b[1][1:], out=out[1:38])
    assert torch.equal(out[1:38], whole[3:, 1:])
    assert bool((out[0] == -7).all()) and bool((out[38:] == -7).all())
    with pytest.raises(ValueError):
        mm.mxfp4_gemm(a[0][:, :16].repeat(1, 2)[:, ::2], a[1], *b)      # not contiguous
    with pytest.raises(ValueError):
        mm.mxfp4_gemm(*a, b[0], b[1][:5])
    with pytest.raises(TypeError):
        mm.mxfp4_gemm(*a, *b, dtype=torch.bfloat16, out=out[:40])


def _dev_mx(shape, K, seed, lo=124, hi=127):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randint(0, 256, (*shape, K // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(lo, hi + 1, (*shape, K // 32), dtype=torch.uint8, device=DEV, generator=g)]


def _rows(pair, rows):
    return [v[rows].cpu().numpy() for v in pair]


def test_gemm_offsets_past_32_bits(mm):
    say("gemm: 8.6 GB of output, then 6.9 GB of codes")
    a, b = _dev_mx((66000,), 32, 1), _dev_mx((32800,), 32, 2)
    got = mm.mxfp4_gemm(*a, *b)
    rows = [0, 16383, 32767, 33000, 65535, 65999]
    want, _ = oa4.gemm(*_rows(a, rows), *[v.cpu().numpy() for v in b])
    assert np.array_equal(got[rows].cpu().numpy().astype(np.float64), want)
    del got, a, b
    a, b = _dev_mx((210000,), 65536, 3, 126, 127), _dev_mx((20,), 65536, 4, 126, 126)
    rows = [0, 131072, 131073, 209999]
    want, mag = oa4.gemm(*_rows(a, rows), *[v.cpu().numpy() for v in b])
    got = mm.mxfp4_gemm(*a, *b)[rows].cpu().numpy()
    assert np.all(np.abs(got - want) <= sum_bound(65536, mag))
    wide = mm.mxfp4_gemm(*b, *a)[:, rows].cpu().numpy()     # as the weights' side
    assert np.all(np.abs(wide.T - want) <= sum_bound(65536, mag))


# ---- grouped --------------------------------------------------------------------

GROUPED = [  # T, H, I, E, k, how the ids are drawn
    (1, 32, 32, 1, 1, "uniform"), (1, 64, 96, 4, 4, "uniform"), (5, 96, 32, 7, 2, "uniform"),
    (8, 256, 128, 8, 2, "dropped"), (70, 160, 64, 3, 2, "uniform"), (300, 512, 160, 4, 3, "skewed"),
    (64, 2048, 256, 16, 4, "uniform"), (40, 64, 64, 1024, 32, "uniform"), (600, 256, 256, 2, 1, "skewed"),
    (20, 1056, 352, 24, 3, "dropped"), (400, 1024, 512, 5, 2, "skewed"), (9, 2048, 2048, 6, 2, "uniform"),
    (700, 512, 288, 3, 2, "uniform"),
]


def lists(rng, T, E, k, how):
    p = np.ones(E) if how != "skewed" else np.arange(1, E + 1, dtype=float) ** -2.0
    ids = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)
    if how == "dropped":
        ids[rng.random((T, k)) < 0.3] = -1
    flat = ids.ravel()
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable").astype(np.int32)
    n = int((flat >= 0).sum())
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]).astype(np.int32)
    order[n:] = -1                                  # what lies past the last segment is not read
    return order, offsets, n


def scale_lo(K):
    return 124 if K <= 1280 else 126


@pytest.mark.parametrize("T,H,I,E,k,how", GROUPED)
def test_gate_up(mm, T, H, I, E, k, how):
    say("gate_up", T, H, I, E, k, how)
    rng = np.random.default_rng(T + H + I)
    pairs, offsets, n = lists(rng, T, E, k, how)
    lo = scale_lo(H)
    x, w = mx(rng, (T,), H, lo), mx(rng, (E, 2 * I), H, lo - 8, 119)
    g, u, _, _ = oa4.gate_up(*x, pairs, offsets, k, *w)
    want = oa4.silu(g) * u
    h = torch.full((T * k, I), -7.0, dtype=torch.bfloat16, device=DEV)
    args = [*up(x), torch.from_numpy(pairs).to(DEV), torch.from_numpy(offsets).to(DEV), k, *up(w)]
    mm.moe_mxfp4_a4_gate_up_swiglu(*args, h=h)
    got = omx.bf16_bits_to_f64(host_bits(h))
    assert np.all(got[n:] == -7.0)
    tol = (2.0 ** -8 + 2.0 ** -21 * (2 + np.abs(g))) * np.abs(want) + 2.0 ** -126
    assert np.all(np.abs(got[:n] - want) <= tol)
    # the packed form holds mxfp4_pack of the same h
    hc = torch.full((T * k, I // 2), 0x5a, dtype=torch.uint8, device=DEV)
    hs = torch.full((T * k, I // 32), 0x5a, dtype=torch.uint8, device=DEV)
    mm.moe_mxfp4_a4_gate_up_swiglu_pack(*args, h_codes=hc, h_scales=hs)
    if n:
        pc, ps = mm.mxfp4_pack(h[:n].contiguous())
        assert torch.equal(hc[:n], pc) and torch.equal(hs[:n], ps)
    assert bool((hc[n:] == 0x5a).all()) and bool((hs[n:] == 0x5a).all())


@pytest.mark.parametrize("T,H,I,E,k,how", GROUPED)
def test_down(mm, T, H, I, E, k, how):
    say("down", T, H, I, E, k, how)
    rng = np.random.default_rng(T + H + I + 1)
    _, offsets, n = lists(rng, T, E, k, how)
    lo = scale_lo(I)
    h, w = mx(rng, (T * k,), I, lo), mx(rng, (E, H), I, lo)
    want, _ = oa4.down(*h, offsets, *w)
    y = torch.full((T * k, H), -7.0, device=DEV)
    mm.moe_mxfp4_a4_down(*up(h), torch.from_numpy(offsets).to(DEV), k, *up(w), y=y)
    got = y.cpu().numpy().astype(np.float64)
    assert np.all(got[n:] == -7.0)
    assert np.array_equal(got[:n], want)


def test_gate_up_special_values(mm):
    """A NaN token gives NaN rows and NaN blocks; overflowing gates keep silu's limits."""
    say("gate_up specials")
    rng = np.random.default_rng(9)
    T, H, I, E, k = 40, 256, 64, 3, 1
    pairs, offsets, n = lists(rng, T, E, k, "uniform")
    x, w = mx(rng, (T,), H), mx(rng, (E, 2 * I), H, 116, 119)
    x[1][3, 2] = 255
    x[1][5, :] = 160                                 # gates near +-2^40
    args = [*up(x), torch.from_numpy(pairs).to(DEV), torch.from_numpy(offsets).to(DEV), k, *up(w)]
    h = mm.moe_mxfp4_a4_gate_up_swiglu(*args)
    got = omx.bf16_bits_to_f64(host_bits(h))
    g, u, _, _ = oa4.gate_up(*x, pairs, offsets, k, *w)
    with np.errstate(over="ignore"):
        want = oa4.silu(g) * u
    bad = pairs[:n] // k == 3
    assert np.isnan(got[bad]).all() and not np.isnan(got[~bad]).any()
    big = pairs[:n] // k == 5
    # a large negative gate gives -0 (its exponential overflows), a positive one g u
    assert np.all(np.abs(got[big] - want[big]) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want[big]) + 1e-30)
    hc, hs = mm.moe_mxfp4_a4_gate_up_swiglu_pack(*args)
    pc, ps = mm.mxfp4_pack(h)
    assert torch.equal(hc, pc) and torch.equal(hs, ps)
    assert bool((hs.cpu().numpy()[bad] == 255).all())


# ---- the layer ---------------------------------------------------------------------

def _layer_inputs(T, H, I, E, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, device=DEV, generator=g)
    return x, logits, _dev_mx((E, 2 * I), H, seed + 1, 118, 124), _dev_mx((E, H), I, seed + 2, 118, 124)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (16, 256, 128, 8, 2), (200, 512, 256, 6, 3),
                                       (33, 96, 160, 5, 5), (2048, 256, 128, 384, 8)])
def test_layer_is_its_calls(mm, T, H, I, E, k):
    say("a4 layer", T, H, I, E, k)
    x, logits, w13, w2 = _layer_inputs(T, H, I, E, T)
    b = mm.moe_mxfp4_a4_layer(x, logits, k, *w13, *w2)
    ids, tw, counts, offsets, pairs, p2r = mm.moe_route_permute(logits, k)
    xq = mm.mxfp4_pack(x)
    hq = mm.moe_mxfp4_a4_gate_up_swiglu_pack(*xq, pairs, offsets, k, *w13)
    y = mm.moe_mxfp4_a4_down(*hq, offsets, k, *w2)
    out = mm.moe_combine(y, tw, p2r)
    for name, want in (("topk_ids", ids), ("topk_w", tw), ("counts", counts), ("offsets", offsets),
                       ("sorted_pairs", pairs), ("pair_to_row", p2r), ("x_codes", xq[0]),
                       ("x_scales", xq[1]), ("h_codes", hq[0]), ("h_scales", hq[1]), ("y", y), ("out", out)):
        assert torch.equal(getattr(b, name), want), name
    # against the oracle, stage by stage: y from the GPU's own h, h from x
    if T > 300:
        return
    host = lambda ts: [t.cpu().numpy() for t in ts]  # noqa: E731
    yo, mag = oa4.down(*host(hq), offsets.cpu().numpy(), *host(w2))
    assert np.all(np.abs(y.cpu().numpy() - yo) <= sum_bound(I, mag))
    g, u, _, _ = oa4.gate_up(*host(xq), pairs.cpu().numpy(), offsets.cpu().numpy(), k, *host(w13))
    hc, hs = omx.pack(omx.bf16_bits_to_f64(omx.to_bf16_bits(oa4.silu(g) * u)))
    # h may round to the neighbouring bf16 where it lies within 2^-18 of a
    # midpoint (one in 2^10); the code changes only if that neighbour is on the
    # other side of one of the 15 thresholds, and a block's 32 codes when its
    # largest element crosses a power of two
    assert (hs != hq[1].cpu().numpy()).mean() <= 2.0 ** -8
    assert (hc != hq[0].cpu().numpy()).mean() <= 2.0 ** -7


def test_layer_page_shaped(mm):
    """The page-shaped layer: 4.8 GB of gate/up codes.  Sampled rows of h and y
    of every kernel path, first and last experts among them, against the
    oracle applied to the GPU's own inputs of that stage."""
    H, I, E, k = 6144, 2048, 384, 8
    w13, w2 = _dev_mx((E, 2 * I), H, 5, 118, 124), _dev_mx((E, H), I, 6, 118, 124)
    for T in (1, 8, 64, 512, 1500):
        say("a4 page-shaped layer, T", T)
        g = torch.Generator(device=DEV).manual_seed(T)
        x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
        rank = torch.arange(1, E + 1, device=DEV).float()
        logits = 1.5 * torch.randn(T, E, device=DEV, generator=g)
        if T == 512:
            logits = logits - 1.1 * rank.flip(0).log()
        b = mm.A4LayerBuffers(T, H, I, E, k, DEV)
        b.y.fill_(float("nan"))
        b.out.fill_(float("nan"))
        mm.moe_mxfp4_a4_layer(x, logits, k, *w13, *w2, buffers=b)
        assert bool(torch.isfinite(b.y).all()) and bool(torch.isfinite(b.out).all())
        h = mm.moe_mxfp4_a4_gate_up_swiglu(b.x_codes, b.x_scales, b.sorted_pairs, b.offsets, k, *w13)
        pc, ps = mm.mxfp4_pack(h)
        assert torch.equal(pc, b.h_codes) and torch.equal(ps, b.h_scales)
        off = b.offsets.cpu().numpy()
        pairs = b.sorted_pairs.cpu().numpy()
        rng = np.random.default_rng(T)
        live = np.flatnonzero(np.diff(off))
        for e in {live[0], live[-1], int(np.argmax(np.diff(off))), *rng.choice(live, 3)}:
            rows = np.unique([off[e], off[e + 1] - 1, rng.integers(off[e], off[e + 1])])
            xs = _rows((b.x_codes, b.x_scales), pairs[rows] // k)
            w = [v[e].cpu().numpy() for v in w13]
            gu, _ = oa4.gemm(*xs, *w)
            want = oa4.silu(gu[:, :I]) * gu[:, I:]
            got = omx.bf16_bits_to_f64(host_bits(h[rows]))
            tol = (2.0 ** -8 + 2.0 ** -21 * (2 + np.abs(gu[:, :I]))) * np.abs(want)
            # these sums are exact too: weights of 2^-9 .. 2^-3 on normal tokens
            assert np.all(np.abs(got - want) <= tol + 2.0 ** -100), e
            hs = _rows((b.h_codes, b.h_scales), rows)
            yo, mag = oa4.gemm(*hs, *[v[e].cpu().numpy() for v in w2])
            assert np.all(np.abs(b.y[rows].cpu().numpy() - yo) <= sum_bound(I, mag)), e


def test_layer_captured_and_on_two_streams(mm):
    say("a4 layer: graph replays and two streams")
    T, H, I, E, k = 40, 512, 256, 6, 2
    x, logits, w13, w2 = _layer_inputs(T, H, I, E, 3)
    x2 = (x * 0.5 + 0.25).contiguous()
    eager = [mm.moe_mxfp4_a4_layer(v, logits, k, *w13, *w2).out.clone() for v in (x, x2)]
    buf = mm.A4LayerBuffers(T, H, I, E, k, DEV)
    xin = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mm.moe_mxfp4_a4_layer(xin, logits, k, *w13, *w2, buffers=buf)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm.moe_mxfp4_a4_layer(xin, logits, k, *w13, *w2, buffers=buf)
    for i in range(4):
        xin.copy_((x, x2)[i % 2])
        buf.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, eager[i % 2]), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [mm.A4LayerBuffers(T, H, I, E, k, DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, bb, v in zip(streams, bufs, (x, x2)):
            with torch.cuda.stream(st):
                mm.moe_mxfp4_a4_layer(v, logits, k, *w13, *w2, buffers=bb)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0].out, eager[0]) and torch.equal(bufs[1].out, eager[1])
    with pytest.raises(ValueError):
        mm.moe_mxfp4_a4_layer(x[:8].contiguous(), logits[:8].contiguous(), k, *w13, *w2, buffers=buf)
