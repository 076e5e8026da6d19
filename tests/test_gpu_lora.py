"""GPU parity of low-rank adapters with the float64 oracle.

Products are exact and a x is carried in fp32 (rounded once more where it is
scaled), then exactly in three bf16 parts, so an element of fp32 y is off by at
most K + 8 roundings of a sum of |a x| carried through |b|, and 3 r + 8 of the
outer sum; each rounding is taken as a whole step, 2^-23, since the matrix
instruction need not round to nearest.  y adds one rounding of its type.  With
small whole numbers every sum is exact and results are required to be equal."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say
from oracle import mx as omx
from oracle import scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def bf16(v):
    """(device tensor, the float64 values it holds)"""
    bits = omx.to_bf16_bits(v)
    return torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).to(DEV), omx.bf16_bits_to_f64(bits)


def store(v, dtype):
    if dtype == torch.bfloat16:
        return bf16(v)
    v = np.asarray(v, np.float32)
    return torch.from_numpy(v).to(DEV), v.astype(np.float64)


def lists(mm, slots, S):
    _, offsets, rows, _ = mm.moe_permute(torch.from_numpy(np.asarray(slots, np.int32)).to(DEV).view(-1, 1), S)
    return rows, offsets


def inputs(rng, M, K, N, S, r, whole):
    if whole:                                             # |t| <= 4 K / 4, sums far below 2^24
        return (rng.integers(-2, 3, (M, K)), rng.integers(-2, 3, (S, r, K)) * (rng.random((S, r, K)) < 0.3),
                rng.integers(-2, 3, (S, N, r)), rng.integers(-8, 9, (M, N)), 2.0 ** rng.integers(-1, 3, S))
    return (rng.normal(size=(M, K)), rng.normal(size=(S, r, K)) / np.sqrt(K), rng.normal(size=(S, N, r)),
            rng.normal(size=(M, N)), rng.random(S) + 0.25)


def check(mm, slots, K, N, S, r, dtype, whole, rng, with_scale=True, **kw):
    M = len(slots)
    x, a, b, y, scale = inputs(rng, M, K, N, S, r, whole)
    scale = scale.astype(np.float32) if with_scale else None
    (xt, x), (at, a), (bt, b), (yt, y) = bf16(x), bf16(a), bf16(b), store(y, dtype)
    rows, offsets = lists(mm, slots, S)
    before = yt.clone()
    got = mm.lora_add(xt, rows, offsets, at, bt, yt, scale=None if scale is None else torch.from_numpy(scale).to(DEV), **kw)
    assert got is yt
    got = yt.double().cpu().numpy()
    want = scored.lora(x, slots, a, b, y, scale)
    bare = np.array([not 0 <= s < S for s in slots], bool)
    assert torch.equal(yt[torch.from_numpy(bare).to(DEV)], before[torch.from_numpy(bare).to(DEV)])
    if whole:
        want = store(want, dtype)[1]                      # exact in fp32, rounded once to bf16
        assert np.array_equal(got, want)
        return
    full, outer = scored.lora_magnitudes(x, slots, a, b, scale)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -9 * (1 + 2.0 ** -8)
    tol = 2.0 ** -23 * ((K + 8) * full + (3 * r + 8) * outer) + 2.0 ** -24 * np.abs(want)
    tol += 2 * half * (np.abs(want) + tol)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / np.maximum(tol, 1e-300))


# M, K, N, S, r, rows an adapter gets in a run
SHAPES = [(1, 8, 1, 1, 1, 1), (1, 2048, 256, 4, 8, 1), (7, 40, 5, 3, 7, 2), (8, 6144, 384, 8, 16, 8), (16, 256, 64, 1, 16, 16),
          (17, 264, 65, 2, 8, 17), (33, 520, 100, 5, 13, 6), (64, 1352, 1001, 7, 24, 5), (65, 1024, 63, 64, 32, 1),
          (100, 72, 130, 3, 33, 40), (130, 2056, 258, 2, 64, 70), (300, 512, 96, 4, 64, 128), (257, 384, 200, 2, 128, 150),
          (90, 136, 72, 9, 100, 3), (513, 128, 40, 6, 5, 100), (40, 4096, 31, 1024, 4, 1), (600, 96, 48, 1, 16, 600),
          (3, 16, 2000, 2, 16, 1), (20, 8, 8, 2, 128, 4), (1000, 32, 24, 30, 48, 40)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_oracle(mm, shape, dtype):
    M, K, N, S, r, run = shape
    say("lora_add", shape, dtype)
    rng = np.random.default_rng(list(shape))
    slots = np.repeat(rng.integers(0, S, -(-M // run)), run)[:M]
    check(mm, slots, K, N, S, r, dtype, True, rng)
    mixed = np.where(rng.random(M) < 0.3, rng.choice([-1, S, 2 ** 30, -2 ** 31], M), rng.integers(0, S, M))
    check(mm, mixed, K, N, S, r, dtype, True, rng, with_scale=False)
    check(mm, slots, K, N, S, r, dtype, False, rng)
    check(mm, mixed, K, N, S, r, dtype, False, rng)


def test_no_row_has_an_adapter(mm):
    say("lora_add without adapters")
    rng = np.random.default_rng(1)
    for M in (1, 50):
        check(mm, np.full(M, -1), 64, 40, 3, 8, torch.float32, False, rng)


def test_unlike_adapters(mm):
    """One row, hundreds of rows and no row side by side."""
    say("lora_add unlike adapters")
    rng = np.random.default_rng(2)
    slots = rng.permutation(np.concatenate([np.full(400, 3), [0, 5, 5], np.full(17, 6), np.full(31, 2), [-1] * 9]))
    for r in (8, 16, 64):
        for dtype in (torch.float32, torch.bfloat16):
            check(mm, slots, 328, 150, 8, r, dtype, True, rng)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_unaligned_y_and_its_neighbours(mm, dtype):
    """y at any element's address; what lies around its rows stays."""
    say("lora_add unaligned", dtype)
    rng = np.random.default_rng(3)
    for N in (16, 64, 72, 200):
        for shift in (0, 1, 3):
            M, K, S, r = 21, 64, 2, 8
            x, a, b, y, _ = inputs(rng, M, K, N, S, r, True)
            (xt, x), (at, a), (bt, b) = bf16(x), bf16(a), bf16(b)
            flat = torch.full((M * N + 64,), 77.0, dtype=dtype, device=DEV)
            yt = flat[shift:shift + M * N].view(M, N)
            yt.copy_(torch.from_numpy(y.astype(np.float32)))
            slots = rng.integers(-1, S, M)
            mm.lora_add(xt, *lists(mm, slots, S), at, bt, yt)
            want = store(scored.lora(x, slots, a, b, y), dtype)[1]
            assert np.array_equal(yt.double().cpu().numpy(), want)
            assert (flat[:shift] == 77.0).all() and (flat[shift + M * N:] == 77.0).all()


def test_infinities_and_nan_stay_in_their_rows(mm):
    say("lora_add infinities")
    rng = np.random.default_rng(4)
    M, K, N, S, r = 40, 64, 70, 3, 13
    x, a, b, y, _ = inputs(rng, M, K, N, S, r, False)
    slots = rng.integers(0, S, M)
    slots[:6] = [0, 1, 2, 0, 1, -1]
    a[:, :, :2], b = np.abs(a[:, :, :2]) + 1.0, np.abs(b) + 0.1
    x[0, 0], x[1, 1], x[2, 0], x[3, 1], x[5] = np.inf, -np.inf, np.nan, 3e38, np.nan
    (xt, x), (at, a), (bt, b), (yt, y) = bf16(x), bf16(a), bf16(b), store(y, torch.float32)
    x = np.where(np.abs(x) < 1e39, x, 0)
    mm.lora_add(xt, *lists(mm, slots, S), at, bt, yt)
    got = yt.double().cpu().numpy()
    assert (got[0] == np.inf).all() and (got[1] == -np.inf).all() and np.isnan(got[2]).all()
    assert not np.isnan(got[3]).any()
    assert np.array_equal(got[5], y[5])
    x[3] = 0
    want = scored.lora(x, slots, a, b, y)
    rest = [m for m in range(M) if m not in (0, 1, 2, 3, 5)]
    assert np.abs(got[rest] - want[rest]).max() <= 1e-4 * np.abs(want[rest]).max()


def test_adapters_of_other_rows_do_not_leak(mm):
    """NaN in one adapter reaches its own rows alone, also where a tile ends early."""
    say("lora_add leaks")
    rng = np.random.default_rng(6)
    slots = np.array([0] * 3 + [1] * 20 + [2] * 5 + [-1] * 2)
    x, a, b, y, _ = inputs(rng, 30, 48, 90, 3, 12, True)
    (xt, x), (at, a), (bt, b), (yt, y) = bf16(x), bf16(a), bf16(b), store(y, torch.float32)
    at[1], bt[1] = float("nan"), float("nan")
    mm.lora_add(xt, *lists(mm, slots, 3), at, bt, yt)
    got = yt.double().cpu().numpy()
    b[1] = a[1] = 0
    want = scored.lora(x, slots, a, b, y)
    assert np.isnan(got[3:23]).all()
    assert np.array_equal(got[:3], want[:3]) and np.array_equal(got[23:], want[23:])


def test_workspace_streams_replays_and_refusals(mm):
    say("lora_add buffers, streams, replays")
    rng = np.random.default_rng(7)
    for M, K, N, S, r in ((8, 512, 100, 2, 8), (200, 256, 130, 5, 24), (40, 264, 72, 3, 100)):
        x, a, b, y, scale = inputs(rng, M, K, N, S, r, False)
        (xt, _), (at, _), (bt, _), (yt, _) = bf16(x), bf16(a), bf16(b), store(y, torch.float32)
        sc = torch.from_numpy(scale.astype(np.float32)).to(DEV)
        slots = [rng.integers(-1, S, M) for _ in range(3)]
        sets = [lists(mm, s, S) for s in slots]
        want = [mm.lora_add(xt, *s, at, bt, yt.clone(), scale=sc) for s in sets]
        again = mm.lora_add(xt, *sets[0], at, bt, yt.clone(), scale=sc)
        assert torch.equal(again, want[0])                 # deterministic
        ws = torch.full((mm.lora_add_workspace_bytes(M, K, N, S, r),), 0xff, dtype=torch.uint8, device=DEV)
        out, rows, offsets = yt.clone(), sets[0][0].clone(), sets[0][1].clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            mm.lora_add(xt, rows, offsets, at, bt, out, scale=sc, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mm.lora_add(xt, rows, offsets, at, bt, out, scale=sc, workspace=ws)
        for i in range(5):
            rows.copy_(sets[i % 3][0])
            offsets.copy_(sets[i % 3][1])
            out.copy_(yt)
            ws.fill_(0xff)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i % 3]), i
    with pytest.raises(mm._lib.MxmError):
        mm.lora_add(xt, *sets[0], at, bt, yt, workspace=ws[:-1])
    with pytest.raises(ValueError):
        mm.lora_add(xt, *sets[0], at, bt[:, :, :8], yt)
    with pytest.raises(ValueError):
        mm.lora_add(xt, *sets[0], at, bt, yt[:, ::2])
    with pytest.raises(TypeError):
        mm.lora_add(xt.float(), *sets[0], at, bt, yt)
    with pytest.raises(mm._lib.MxmError):                  # K no multiple of 8
        mm.lora_add(xt[:, :12].contiguous(), *sets[0], at[:, :, :12].contiguous(), bt, yt)
    empty = mm.lora_add(xt[:0], sets[0][0][:0], sets[0][1], at, bt, yt[:0])
    assert empty.shape == (0, yt.shape[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_zero_adapters_keep_every_value(mm, dtype):
    """y + 0 is y, for the smallest and largest numbers of its type too."""
    say("lora_add of nothing", dtype)
    g = torch.Generator(device=DEV).manual_seed(1)
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    top = 0x7f80 if dtype == torch.bfloat16 else 0x7f800000
    for M, r in ((40, 16), (40, 100)):
        mag = torch.randint(0, top, (M, 96), device=DEV, generator=g)      # every finite magnitude
        mag[:, :48] = mag[:, :48] >> 8                                      # half of them tiny or subnormal
        sign = torch.where(torch.rand(M, 96, device=DEV, generator=g) < 0.5, -1, 1).to(dtype)
        y = mag.to(bits).view(dtype) * sign
        before = y.clone()
        x = torch.randn(M, 64, device=DEV, generator=g).bfloat16()
        a, b = torch.zeros(2, r, 64, dtype=torch.bfloat16, device=DEV), torch.ones(2, 96, r, dtype=torch.bfloat16, device=DEV)
        mm.lora_add(x, *lists(mm, np.arange(M) % 2, 2), a, b, y)
        assert torch.equal(y, before)


def test_more_than_2_to_32_elements_of_y(mm):
    say("lora_add past 32 bits")
    M, K, N, S, r = 270000, 8, 16384, 2, 8
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randint(-2, 3, (M, K), device=DEV, generator=g).bfloat16()
    a = torch.randint(-2, 3, (S, r, K), device=DEV, generator=g).bfloat16()
    b = torch.randint(-2, 3, (S, N, r), device=DEV, generator=g).bfloat16()
    y = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    assert y.numel() > 2 ** 32
    slots = torch.randint(-1, S, (M, 1), device=DEV, generator=g).int()
    _, offsets, rows, _ = mm.moe_permute(slots, S)
    mm.lora_add(x, rows, offsets, a, b, y)
    for m in (0, 1, 131071, 131072, 262143, 262144, M - 2, M - 1):
        s = int(slots[m])
        want = torch.zeros(N, device=DEV) if s < 0 else b[s].float() @ (a[s].float() @ x[m].float())
        assert torch.equal(y[m], want.bfloat16()), m


def test_two_calls_at_once(mm):
    """Two streams, a workspace each, the same inputs."""
    say("lora_add on two streams")
    rng = np.random.default_rng(10)
    M, K, N, S, r = 96, 1024, 640, 3, 100
    x, a, b, y, scale = inputs(rng, M, K, N, S, r, False)
    (xt, _), (at, _), (bt, _), (yt, _) = bf16(x), bf16(a), bf16(b), store(y, torch.bfloat16)
    ll = lists(mm, rng.integers(-1, S, M), S)
    want = mm.lora_add(xt, *ll, at, bt, yt.clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    nws = mm.lora_add_workspace_bytes(M, K, N, S, r)
    assert nws > 0
    ws = [torch.empty(nws, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [[yt.clone() for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                mm.lora_add(xt, *ll, at, bt, outs[j][i], workspace=ws[j])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for side in outs for o in side)


def test_projection_router_and_routing_together(mm):
    """Rows of several requests: the shared product in MXFP4, the adapters beside it, the
    adapted router's logits, and the experts of each token from them."""
    say("projection, adapters, router and routing")
    rng = np.random.default_rng(9)
    M, K, N, S, r, E = 48, 256, 192, 4, 16, 32
    slots = np.repeat([0, 2, -1, 3, 1, 2], 8)
    xt, x = bf16(rng.normal(size=(M, K)))
    w = rng.normal(size=(N, K)).astype(np.float32) / 16
    wc, ws = mm.mxfp4_pack(torch.from_numpy(w).to(DEV))
    xc, xs = mm.mxfp4_pack(xt)
    base = mm.mxfp4_gemm(xc, xs, wc, ws)
    (at, a), (bt, b) = bf16(rng.normal(size=(S, r, K)) / 16), bf16(rng.normal(size=(S, N, r)) / 4)
    rows, offsets = lists(mm, slots, S)
    x64, w64 = (mm.mxfp4_unpack(c, s).double().cpu().numpy() for c, s in ((xc, xs), (wc, ws)))
    got = mm.lora_add(xt, rows, offsets, at, bt, base).double().cpu().numpy()
    want = scored.lora(x, slots, a, b, x64 @ w64.T)
    assert np.abs(got - want).max() <= 1e-5 * np.abs(want).max()
    router = rng.normal(size=(E, K)).astype(np.float32) / 16
    logits, _, _ = mm.moe_router_topk(xt, torch.from_numpy(router).to(DEV), 4)
    (ra, ra64), (rb, rb64) = bf16(rng.normal(size=(S, 8, K)) / 16), bf16(rng.normal(size=(S, E, 8)) / 4)
    mm.lora_add(xt, rows, offsets, ra, rb, logits)
    want = scored.lora(x, slots, ra64, rb64, x @ router.astype(np.float64).T)
    assert np.abs(logits.double().cpu().numpy() - want).max() <= 1e-5 * np.abs(want).max()
    bias = (rng.integers(-20, 21, E) / 1024).astype(np.float32)
    ids, wt = mm.moe_route_scored(logits, 4, bias=torch.from_numpy(bias).to(DEV), groups=4, topk_groups=2, scale=2.5)
    oid, ow = scored.route(logits.cpu().numpy(), 4, bias, groups=4, keep=2, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), oid)
    assert np.abs(wt.double().cpu().numpy() - ow).max() <= 2.0 ** -18 * 2.5


# thousands of rows: tiles of 17 to 48 rows, of a multiple of 16 where those fit, one round and more
HEIGHTS = [(4500, 72, 70, 3, 8), (6000, 40, 33, 20, 5), (8192, 64, 68, 8, 16), (8300, 40, 132, 5, 64), (12000, 48, 40, 60, 33),
           (20000, 32, 36, 9, 30), (9000, 24, 64, 300, 16), (10100, 16, 4100, 3, 24)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", HEIGHTS, ids=lambda s: "x".join(map(str, s)))
def test_tile_heights(mm, shape, dtype):
    M, K, N, S, r = shape
    say("lora_add tile heights", shape, dtype)
    rng = np.random.default_rng(list(shape))
    even = np.arange(M) * S // M
    check(mm, even, K, N, S, r, dtype, True, rng)
    check(mm, np.where(rng.random(M) < 0.02, -1, rng.integers(0, S, M)), K, N, S, r, dtype, True, rng)
    check(mm, np.zeros(M, int), K, N, S, r, dtype, False, rng)
    check(mm, np.minimum(rng.geometric(0.4, M) - 1, S - 1), K, N, S, r, dtype, False, rng)
