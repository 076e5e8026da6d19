"""Low-rank adapters in both of their forms, one launch and two, at every padded
rank, and the 24 bits of t = A x.

Which form a call takes shows in its workspace: none for one launch, and for two
[pieces of K, rows, padded rank] of fp32."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say
from oracle import scored
from test_gpu_lora import bf16, check, lists, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


# M, K, N, S, r, padded rank, pieces of K; rows in tiles of 16 and, from 32 an
# adapter on, of 32; r and N of whole vectors and not; last pieces that are short
# (K 1000, 2056) or empty (1032, 2056, 4104)
TWO = [(3, 8456, 40, 2, 8, 8, 16), (2, 8456, 37, 1, 5, 8, 16), (70, 8456, 44, 2, 8, 8, 16), (33, 8200, 37, 1, 5, 8, 16),
       (3, 8456, 40, 2, 16, 16, 16), (5, 8264, 66, 3, 13, 16, 16), (64, 8456, 36, 1, 16, 16, 16), (66, 8200, 35, 2, 11, 16, 16),
       (4, 5472, 44, 2, 32, 32, 16), (5, 6144, 66, 2, 24, 32, 16), (80, 6144, 68, 2, 24, 32, 16), (64, 5472, 45, 1, 31, 32, 16),
       (8, 6144, 200, 2, 64, 64, 16), (6, 3288, 61, 3, 50, 64, 8), (100, 3288, 60, 3, 64, 64, 8), (90, 3320, 61, 2, 37, 64, 8),
       (9, 488, 36, 2, 128, 128, 1), (7, 1000, 65, 2, 100, 128, 2), (40, 1032, 40, 1, 128, 128, 4), (96, 1024, 640, 3, 100, 128, 4),
       (64, 2056, 37, 2, 128, 128, 8), (5, 4104, 36, 1, 104, 128, 16), (700, 1032, 33, 90, 65, 128, 4), (8200, 64, 36, 200, 128, 128, 1),
       (1040, 520, 300, 130, 72, 128, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", TWO, ids=lambda s: "x".join(map(str, s[:5])))
def test_two_launches_match_oracle(mm, shape, dtype):
    M, K, N, S, r, rank, pieces = shape
    say("lora_add in two launches", shape, dtype)
    assert mm.lora_add_workspace_bytes(M, K, N, S, r) == 4 * pieces * M * rank
    rng = np.random.default_rng([M, K, N, S, r])
    ws = torch.full((4 * pieces * M * rank,), 0xff, dtype=torch.uint8, device=DEV)
    even = np.arange(M) * S // M
    mixed = np.where(rng.random(M) < 0.2, -1, rng.integers(0, S, M))
    check(mm, even, K, N, S, r, dtype, True, rng, workspace=ws)
    check(mm, mixed, K, N, S, r, dtype, True, rng, with_scale=False, workspace=ws)
    check(mm, mixed, K, N, S, r, dtype, False, rng, workspace=ws)


# M, K, N, S, r, two launches; in one launch tiles of 16, 17 to 32 and 33 to 48 rows
WIDE = [(5, 8456, 40, 2, 8, True), (64, 8456, 37, 1, 7, True), (6, 8456, 40, 3, 16, True), (70, 8264, 41, 2, 13, True),
        (5, 5472, 68, 2, 32, True), (80, 5472, 67, 2, 27, True), (7, 3288, 132, 3, 64, True), (66, 3288, 131, 2, 61, True),
        (7, 1032, 260, 2, 128, True), (64, 2056, 259, 2, 101, True), (300, 64, 256, 1, 128, True),
        (9, 64, 40, 2, 8, False), (30, 96, 37, 2, 7, False), (17, 2048, 36, 1, 16, False), (40, 520, 50, 5, 13, False),
        (33, 1352, 70, 3, 32, False), (20, 264, 65, 4, 29, False), (50, 1024, 136, 2, 64, False), (21, 136, 131, 2, 61, False),
        (6000, 64, 36, 3, 8, False), (5000, 40, 50, 9, 13, False), (6000, 48, 64, 3, 32, False), (6000, 48, 69, 3, 27, False),
        (6000, 40, 132, 3, 64, False), (5500, 40, 67, 40, 61, False),
        # (taller than 32 only where tiles of 32 rows are more than 256)
        (9500, 40, 40, 8, 8, False), (9500, 40, 37, 8, 5, False), (9500, 40, 44, 8, 16, False), (9500, 40, 50, 8, 15, False),
        (9500, 40, 68, 8, 32, False), (9500, 40, 67, 8, 27, False), (9500, 40, 132, 8, 64, False), (9800, 40, 131, 20, 50, False)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "x".join(map(str, s[:5])))
def test_all_24_bits_of_t(mm, shape, dtype):
    """t = 2^16 p + 2^8 q + s with odd p, q and s of eight bits, other ones for each
    rank and adapter: no step may leave out a bit, and with one power of two a column
    of B every sum is exact, so results are required to be equal."""
    M, K, N, S, r, two = shape
    say("lora_add, 24 bits of t", shape, dtype)
    assert (mm.lora_add_workspace_bytes(M, K, N, S, r) > 0) == two
    rng = np.random.default_rng([M, K, N, S, r, 24])
    slots = rng.integers(-1, S, M)
    part = 2 * rng.integers(0, 128, (S, r, 3)) + 1        # p, q, s
    at = np.array([rng.choice(K, 3, replace=False) for _ in range(S)])
    a = rng.integers(-5, 6, (S, r, K))
    x = np.zeros((M, K))
    power, sign = 2.0 ** rng.integers(-6, 7, M), rng.choice([-1.0, 1.0], M)
    for s in range(S):
        a[s][:, at[s]] = part[s]
        rows = np.flatnonzero(slots == s)
        x[rows[:, None], at[s]] = (power * sign)[rows, None] * np.array([65536.0, 256.0, 1.0])
    rank = np.stack([rng.permutation(np.arange(N) % r) for _ in range(S)])          # of each column
    factor = rng.choice([-1.0, 1.0], (S, N)) * 2.0 ** rng.integers(-3, 4, (S, N))
    b = np.zeros((S, N, r))
    np.put_along_axis(b, rank[:, :, None], factor[:, :, None], 2)
    scale = (2.0 ** rng.integers(-2, 3, S)).astype(np.float32)
    t = part @ np.array([65536, 256, 1])                  # [S, r]
    assert (t % 256).all() and (t // 256 % 256).all() and t.max() < 2 ** 24
    want = np.zeros((M, N))
    for s in range(S):
        rows = slots == s
        want[rows] = (power * sign)[rows, None] * (float(scale[s]) * factor[s] * t[s][rank[s]])[None]
    yt = torch.zeros(M, N, dtype=dtype, device=DEV)
    mm.lora_add(bf16(x)[0], *lists(mm, slots, S), bf16(a)[0], bf16(b)[0], yt, scale=torch.from_numpy(scale).to(DEV))
    assert np.array_equal(yt.double().cpu().numpy(), store(want, dtype)[1])


def test_two_calls_at_once(mm):
    """Two streams with a workspace each, in two launches with four pieces of K, against
    the oracle, of whole numbers."""
    say("lora_add on two streams, oracle")
    rng = np.random.default_rng(11)
    M, K, N, S, r = 96, 1024, 640, 3, 100
    x, a, b = rng.integers(-2, 3, (M, K)), rng.integers(-2, 3, (S, r, K)), rng.integers(-2, 3, (S, N, r))
    y = rng.integers(-8, 9, (M, N))
    slots = rng.integers(-1, S, M)
    want = scored.lora(x, slots, a, b, y)
    (xt, _), (at, _), (bt, _), (yt, _) = bf16(x), bf16(a), bf16(b), store(y, torch.float32)
    ll = lists(mm, slots, S)
    nws = mm.lora_add_workspace_bytes(M, K, N, S, r)
    assert nws == 4 * 4 * M * 128
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.full((nws,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [[yt.clone() for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                mm.lora_add(xt, *ll, at, bt, outs[j][i], workspace=ws[j])
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert np.array_equal(o.double().cpu().numpy(), want)
