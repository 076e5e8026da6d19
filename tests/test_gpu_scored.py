"""GPU parity of routing by scores with the float64 oracle.

Choices compare values of 64 bits on both sides: two values c that are not equal
are further apart here than fp64 rounds (2^-52), so ids are required to be equal.
Weights: the rule's to 2^-18 relative, the stated bound.  In units of 2^-24: an
exponential is off by 2.5 (its instruction by a unit in the last place, 2^-23, and
its argument's rounding), a score by 6 (two exponentials, a sum, a quotient), a
renormalised weight by twice that, 5 additions, a quotient and a product: 19; a
softmax's by 2.5 and its sum's 2.5 and up to 36 additions, a quotient and a
product: 43 at most, below 64.  Where they leave fp32's normal range they are within
2^-148."""

import numpy as np
import pytest
import torch

import workloads
from _gpu import DEV, dev_bf16, dev_u8, say, tol_check
from oracle import layer as olayer
from oracle import permute as operm
from oracle import scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def up(v):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(DEV)


def weights_match(got, want):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.all(np.abs(got - want) <= 2.0 ** -18 * np.abs(want) + 2.0 ** -148)


def check(mm, logits, k, bias=None, **rule):
    names = {"sigmoid": "score", "keep": "topk_groups", "best": "group_best", "norm": "renormalise"}
    call = {names.get(n, n): v for n, v in rule.items()}
    call["score"] = "sigmoid" if rule.get("sigmoid", True) else "softmax"
    ids, w = scored.route(logits, k, bias, **rule)
    T, E = logits.shape
    got = mm.moe_route_scored(up(logits), k, bias=up(bias), **call)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    weights_match(got[1].cpu().numpy(), w)
    lists = mm.moe_route_scored_permute(up(logits), k, bias=up(bias), **call)
    assert torch.equal(lists[0], got[0]) and torch.equal(lists[1], got[1])
    n = int((ids >= 0).sum())
    want = mm.moe_permute(got[0], E)
    for i, name in enumerate(("counts", "offsets", "sorted_pairs", "pair_to_row")):
        a, b = lists[2 + i].cpu().numpy(), want[i].cpu().numpy()
        if name == "sorted_pairs":
            a, b = a[:n], b[:n]                           # what is dropped is not listed
        assert np.array_equal(a, b), name
    if n == T * k:
        for key, a in zip(("counts", "offsets", "sorted_pairs", "pair_to_row"), lists[2:]):
            assert np.array_equal(a.cpu().numpy(), operm.permute(ids, E)[key]), key
    return ids, w


# T, E, k, groups, keep, best
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 384, 8, 1, 1, 2), (3, 2, 2, 2, 2, 1), (5, 7, 3, 7, 4, 2), (8, 384, 8, 8, 4, 2),
          (16, 256, 8, 8, 4, 2), (17, 160, 6, 8, 3, 1), (16, 1024, 32, 1, 1, 1), (9, 1024, 32, 64, 9, 2),
          (20, 1023, 8, 33, 5, 2), (20, 1020, 8, 17, 5, 2), (20, 1017, 12, 9, 3, 1), (30, 1023, 8, 3, 2, 2),
          (33, 145, 5, 5, 2, 2), (40, 64, 8, 64, 8, 2), (40, 65, 4, 13, 2, 2), (64, 100, 10, 10, 1, 1),
          (12, 63, 9, 1, 1, 2), (12, 129, 32, 1, 1, 2), (700, 24, 3, 4, 2, 2), (6, 512, 8, 1, 1, 1),
          (6, 513, 8, 1, 1, 1), (11, 390, 16, 30, 11, 2), (1100, 48, 8, 6, 5, 1)]


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_oracle(mm, shape, sigmoid):
    T, E, k, groups, keep, best = shape
    say("route_scored", shape, sigmoid)
    rng = np.random.default_rng(list(shape) + [sigmoid])
    for seed, (use_bias, norm, scale) in enumerate([(True, True, 2.5), (False, True, 1.0), (True, False, 1.0), (False, False, -16.0)]):
        skew = rng.normal(0, 0.7, E)
        logits = (rng.normal(0, 1.5, (T, E)) + skew).astype(np.float32)
        # a bias in steps, as balancing sets it
        bias = (np.round(-60 * skew) / 1024 * (1.0 if sigmoid else 8.0 / E)).astype(np.float32) if use_bias else None
        check(mm, logits, k, bias, sigmoid=sigmoid, groups=groups, keep=keep, best=best, norm=norm, scale=scale)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (4, 2, 2), (8, 5, 1)])
def test_ties(mm, groups, keep, best, sigmoid):
    """Logits of few values and biases of fewer: most places are decided by the index."""
    say("route_scored ties", groups, sigmoid)
    rng = np.random.default_rng([groups, sigmoid])
    for T in (9, 50):
        logits = rng.integers(-1, 2, (T, 96)).astype(np.float32)
        logits[logits == 0] *= rng.choice([-1.0, 1.0], (logits == 0).sum())      # zeros of both signs
        logits[0] = 3.0
        check(mm, logits, 8, None, sigmoid=sigmoid, groups=groups, keep=keep, best=best)
        check(mm, logits, 8, np.zeros(96, np.float32), sigmoid=sigmoid, groups=groups, keep=keep, best=best, norm=False)
        check(mm, logits, 8, rng.integers(0, 2, 96).astype(np.float32) / 4, sigmoid=sigmoid, groups=groups, keep=keep, best=best)


@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (4, 2, 2), (16, 3, 1)])
def test_near_ties(mm, groups, keep, best):
    """Values c that fp32 does not tell apart: sigmoids next to 1, and logits one step apart."""
    say("route_scored near ties", groups)
    rng = np.random.default_rng(groups)
    for T in (7, 40):
        far = (18.0 + rng.permuted(np.tile(np.arange(128), (T, 1)), axis=1) / 32).astype(np.float32)
        step = np.float32(0.5) + rng.permuted(np.tile(np.arange(128), (T, 1)), axis=1).astype(np.float32) * np.float32(2.0 ** -24)
        for logits in (far, step, -far):
            check(mm, logits, 8, np.full(128, 0.25, np.float32), groups=groups, keep=keep, best=best)
            check(mm, logits, 8, None, groups=groups, keep=keep, best=best)
        check(mm, step, 8, np.full(128, 2.0 ** -7, np.float32), sigmoid=False, groups=groups, keep=keep, best=best)
        # a large bias leaves fp32 no digit of the score
        check(mm, step, 8, np.full(128, 1024.0, np.float32), groups=groups, keep=keep, best=best)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
def test_unavailable_and_extreme(mm, sigmoid, norm):
    say("route_scored edges", sigmoid, norm)
    rng = np.random.default_rng(5)
    n, i, low = np.nan, np.inf, np.finfo(np.float32).min
    for T in (14, 30):
        logits = rng.normal(0, 2, (T, 40)).astype(np.float32)
        logits[0] = -i                                    # nothing left
        logits[1] = n
        logits[2, 3:] = -i                                # three left
        logits[3, :37] = n
        logits[4] = low                                   # the lowest number is a number
        logits[5, 1:] = low
        logits[6, 7] = i
        logits[7, [4, 30]] = i
        logits[8] = i
        logits[9] -= 1000.0                               # every score underflows
        logits[10] += 1000.0
        logits[11, ::2], logits[11, 1::2] = -i, low
        logits[12, 10:20] = -i                            # a whole group
        logits[13] = 0.0
        for groups, keep, best in ((1, 1, 1), (4, 2, 2), (4, 1, 1), (20, 7, 2)):
            k = min(6, keep * 40 // groups)
            rule = dict(sigmoid=sigmoid, groups=groups, keep=keep, best=best, norm=norm)
            ids, _ = check(mm, logits, k, None, **rule)
            assert (ids[:2] == -1).all()
            check(mm, logits, k, rng.normal(0, 0.1, 40).astype(np.float32), **rule)
            bias = rng.normal(0, 0.1, 40).astype(np.float32)
            bias[[3, 4, 5, 6]] = n, i, -i, low
            check(mm, logits, k, bias, **rule)


# E, k, groups, keep, best: 8, 16, 24 and 32 experts a lane of the kernel for many tokens, and its limits
LARGE = [(384, 8, 1, 1, 1), (384, 8, 8, 4, 2), (384, 6, 4, 2, 1), (256, 8, 8, 4, 2), (64, 8, 16, 5, 2), (512, 8, 1, 1, 2),
         (120, 1, 2, 1, 1), (20, 5, 5, 3, 2), (508, 7, 1, 1, 1), (8, 8, 1, 1, 1), (260, 3, 13, 4, 2), (390, 8, 1, 1, 1),
         (384, 9, 1, 1, 1), (516, 8, 1, 1, 1)]


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_many_tokens_as_few(mm, shape, sigmoid):
    """Thousands of tokens take the experts that calls of a few take, which the
    oracle holds; rows of every awkward kind stand among ordinary ones.  Each
    side's weights are within 2^-18 of the rule's, and of each other's 2^-17."""
    E, k, groups, keep, best = shape
    say("route_scored many as few", shape, sigmoid)
    rng = np.random.default_rng(list(shape) + [sigmoid, 7])
    T = 5003
    logits = rng.normal(0, 1.5, (T, E)).astype(np.float32)
    odd = rng.permutation(T)[:T // 5]
    logits[odd] = rng.integers(-2, 3, (len(odd), E))                       # ties
    i, n = np.inf, np.nan
    for j, at in enumerate(rng.permutation(T)[:200]):
        kind = j % 8
        if kind == 0:
            logits[at] = -i
        elif kind == 1:
            logits[at, rng.random(E) < 0.9] = n
        elif kind == 2:
            logits[at, rng.integers(0, E)] = i
        elif kind == 3:
            logits[at] -= 1000.0
        elif kind == 4:
            logits[at] = np.finfo(np.float32).min
        elif kind == 5:
            logits[at, :E // 2] = -i
        elif kind == 6:
            logits[at] = 0.5 + rng.permutation(E) * 2.0 ** -24             # one step apart
        else:
            logits[at] += 18.0                                              # sigmoids next to 1
    bias = (rng.integers(-60, 61, E) / (1024 if sigmoid else 1024 * E / 8)).astype(np.float32)
    big = up(logits)
    for b, norm in ((bias, True), (None, True), (bias, False), (None, False)):
        call = dict(bias=up(b), score="sigmoid" if sigmoid else "softmax", groups=groups, topk_groups=keep,
                    group_best=best, renormalise=norm, scale=2.5)
        ids, w = (v.cpu().numpy() for v in mm.moe_route_scored(big, k, **call))
        few = [mm.moe_route_scored(big[s:s + 500].contiguous(), k, **call) for s in range(0, T, 500)]
        assert np.array_equal(ids, np.concatenate([v[0].cpu().numpy() for v in few]))
        other = np.concatenate([v[1].cpu().numpy() for v in few]).astype(np.float64)
        assert np.all(np.abs(w - other) <= 2.0 ** -17 * np.abs(other) + 2.0 ** -147)
    some = rng.permutation(T)[:60]
    want, ww = scored.route(logits[some], k, None, sigmoid, groups, keep, best, False, 2.5)
    assert np.array_equal(ids[some], want)
    weights_match(w[some], ww)
    # logits of no vector's alignment
    flat = torch.empty(T * E + 1, device=DEV)
    flat[1:] = big.view(-1)
    got = mm.moe_route_scored(flat[1:].view(T, E), k, **call)
    assert np.array_equal(got[0].cpu().numpy(), ids)


def test_many_tokens(mm):
    """More tokens than a launch has waves, and both sides of every rule on sizes."""
    say("route_scored many tokens")
    T, g = 300001, torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randn(T, 6, device=DEV, generator=g)
    ids, w = mm.moe_route_scored(logits, 2)
    want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), want)
    s = torch.sigmoid(logits.double()).gather(1, want)
    assert float((w - s / s.sum(1, keepdim=True)).abs().max()) <= 2.0 ** -18
    lists = mm.moe_route_scored_permute(logits, 2)
    assert torch.equal(lists[0], ids) and int(lists[3][-1]) == 2 * T


def test_buffers_streams_and_replays(mm):
    say("route_scored buffers, streams, replays")
    rng = np.random.default_rng(8)
    rule = dict(bias=up(rng.normal(0, 0.1, 96).astype(np.float32)), groups=4, topk_groups=2)
    for T in (8, 40, 2000):
        sets = [up(rng.normal(0, 1.5, (T, 96)).astype(np.float32)) for _ in range(3)]
        want = [[v.clone() for v in mm.moe_route_scored_permute(s, 6, **rule)] for s in sets]
        out = [torch.full_like(v, -9) for v in want[0]]
        names = ("topk_ids", "topk_w", "counts", "offsets", "sorted_pairs", "pair_to_row")
        ws = torch.full((max(4, mm.moe_permute_workspace_bytes(T, 96, 6)),), 0xff, dtype=torch.uint8, device=DEV)
        live = sets[0].clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            got = mm.moe_route_scored_permute(live, 6, **rule, workspace=ws, **dict(zip(names, out)))
        torch.cuda.synchronize()
        assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(out, want[0]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mm.moe_route_scored_permute(live, 6, **rule, workspace=ws, **dict(zip(names, out)))
        for i in range(5):
            live.copy_(sets[i % 3])
            for v in out:
                v.fill_(-9)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i % 3])), (T, i)
    with pytest.raises(mm._lib.MxmError):
        mm.moe_route_scored(sets[0], 6, groups=5)
    with pytest.raises(mm._lib.MxmError):
        mm.moe_route_scored_permute(sets[0], 6, workspace=ws[:8])
    with pytest.raises(ValueError):
        mm.moe_route_scored(sets[0], 6, bias=rule["bias"][:95])
    with pytest.raises(ValueError):
        mm.moe_route_scored(sets[0].t(), 6)
    empty = mm.moe_route_scored_permute(sets[0][:0], 6)
    assert empty[0].shape == (0, 6) and empty[4].numel() == 0


@pytest.fixture(scope="module")
def small_layer():
    cfg = workloads.custom_config("scored", 91, 70, 256, 128, 24, 3)
    w = workloads.all_weights(cfg, 0)
    return cfg, w, [dev_u8(w[n]) for n in ("w13_codes", "w13_scales", "w2_codes", "w2_scales")]


@pytest.mark.parametrize("T", [1, 8, 16, 70])
def test_layer(mm, small_layer, T):
    """The layer is its separate calls, bit for bit, and the oracle's experts
    mixed by the oracle's routing; rows that nothing is left for are zeros."""
    say("scored layer", T)
    cfg, w, dev = small_layer
    c = cfg.with_tokens(T)
    xb = workloads.gen_x_bits(c, 0)
    rng = np.random.default_rng(T)
    logits, bias = rng.normal(0, 1, (T, 24)).astype(np.float32), rng.normal(0, 0.1, 24).astype(np.float32)
    logits[T // 2, 2:] = -np.inf                          # two experts left
    if T > 1:
        logits[T - 1] = np.nan                            # none
    rule = dict(score="sigmoid", groups=4, topk_groups=2, group_best=2, scale=2.5)
    x = dev_bf16(xb)
    b = mm.LayerBuffers(T, c.H, c.I, c.E, c.k, DEV)
    for v in (b.h, b.y, b.out):
        v.fill_(7.0)
    got = mm.moe_mxfp4_scored_layer(x, up(logits), 3, *dev, bias=up(bias), **rule, buffers=b)
    assert got is b
    ids, wt, counts, offsets, pairs, row = mm.moe_route_scored_permute(up(logits), 3, bias=up(bias), **rule)
    n = int(offsets[-1])
    assert n < 3 * T
    h = torch.full_like(b.h, 7.0)
    y = torch.full_like(b.y, 7.0)
    mm.moe_mxfp4_gate_up_swiglu(x, pairs, offsets, 3, dev[0], dev[1], h=h)
    mm.moe_mxfp4_down(h, offsets, 3, dev[2], dev[3], y=y)
    out = mm.moe_combine(y, wt, row)
    for a, e in ((b.h, h), (b.y, y), (b.out, out)):
        assert torch.equal(a, e)
    assert (b.y[n:] == 7.0).all() and (b.h[n:] == 7.0).all()
    oid, ow = scored.route(logits, 3, bias, groups=4, keep=2, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), oid)
    # every expert's output of every token from the oracle's layer: all experts, equal weights
    full = olayer.layer_forward(xb, np.tile(-np.arange(24, dtype=np.float32), (T, 1)), w["w13_codes"], w["w13_scales"],
                                w["w2_codes"], w["w2_scales"], 24)
    each = np.asarray(full["y"], np.float64).reshape(T, 24, c.H)          # slot j holds expert j
    want = sum(ow[:, j, None] * each[np.arange(T), np.maximum(oid[:, j], 0)] for j in range(3))
    tol_check(b.out.cpu().numpy(), want, "scored layer out")
    if T > 1:
        assert not b.out[T - 1].any()


@pytest.mark.parametrize("T,E,groups,keep", [(4096, 384, 8, 4), (4127, 384, 1, 1), (8192, 384, 8, 4), (5000, 12, 1, 1),
                                             (6001, 512, 4, 2), (16384, 64, 1, 1), (16385, 64, 1, 1), (4100, 40, 10, 5)])
def test_lists_of_many_tokens(mm, T, E, groups, keep):
    """k = 8: the routing counts for the grouping.  Some tokens have few experts left, or none."""
    say("route_scored_permute, many tokens", T, E, groups)
    g = torch.Generator(device=DEV).manual_seed(T + E)
    logits = torch.randn(T, E, device=DEV, generator=g)
    logits[::97] = float("-inf")
    logits[5::89, E // 4:] = float("nan")
    logits[7::50] = torch.round(logits[7::50])
    rule = dict(bias=torch.round(torch.randn(E, device=DEV, generator=g) * 30) / 1024, groups=groups, topk_groups=keep)
    ids, w = mm.moe_route_scored(logits, 8, **rule)
    assert (ids == -1).any()
    for ws in (None, torch.full((mm.moe_permute_workspace_bytes(T, E, 8),), 0xff, dtype=torch.uint8, device=DEV)):
        got = mm.moe_route_scored_permute(logits, 8, **rule, workspace=ws)
        want = mm.moe_permute(ids, E)
        n = int(want[1][-1])
        assert torch.equal(got[0], ids) and torch.equal(got[1], w)
        assert torch.equal(got[2], want[0]) and torch.equal(got[3], want[1]) and torch.equal(got[5], want[3])
        assert torch.equal(got[4][:n], want[2][:n])


# both sides of every limit between the grouping's kernels: 8192 and 131072 pairs, 4 experts a token
@pytest.mark.parametrize("T,E,k", [(1024, 384, 8), (1025, 384, 8), (2050, 7, 4), (4097, 1024, 4), (5000, 33, 3), (8192, 384, 8),
                                   (4096, 64, 32), (16384, 384, 8), (16385, 384, 8), (2731, 5, 5), (9001, 1, 1), (2049, 4, 4)])
def test_grouping_of_many_pairs(mm, T, E, k):
    say("permute", T, E, k)
    rng = np.random.default_rng([T, E, k])
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    for kind in range(3):
        if kind == 1:                                     # some dropped
            ids = np.where(rng.random((T, k)) < 0.3, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k)), ids).astype(np.int32)
        elif kind == 2:                                   # all of one expert
            ids[:] = E - 1
        got = [v.cpu().numpy() for v in mm.moe_permute(torch.from_numpy(ids).to(DEV), E)]
        flat = ids.ravel()
        ok = (flat >= 0) & (flat < E)
        pairs = np.flatnonzero(ok)
        pairs = pairs[np.argsort(flat[pairs], kind="stable")]
        counts = np.bincount(flat[ok], minlength=E)
        row = np.full(T * k, -1)
        row[pairs] = np.arange(len(pairs))
        assert np.array_equal(got[0], counts) and np.array_equal(got[1], np.concatenate([[0], np.cumsum(counts)]))
        assert np.array_equal(got[2][:len(pairs)], pairs) and np.array_equal(got[3], row)


def test_values_at_the_end_of_the_range(mm):
    """Scores below fp32's normal range next to biases of their size, and far apart ones without a
    bias' help: what fp64 says."""
    say("route_scored tiny values")
    rng = np.random.default_rng(12)
    for T in (12, 40, 4200):
        logits = (-80.0 - 60.0 * rng.random((T, 64))).astype(np.float32)
        for bias in (np.zeros(64, np.float32), (rng.integers(0, 3, 64) * 2.0 ** -120).astype(np.float32),
                     (rng.integers(0, 5, 64) * 2.0 ** -149).astype(np.float32)):
            some = slice(0, 40)
            for sigmoid in (True, False):
                rule = dict(score="sigmoid" if sigmoid else "softmax", groups=4, topk_groups=2)
                ids, w = mm.moe_route_scored(up(logits), 6, bias=up(bias), **rule)
                want, ww = scored.route(logits[some], 6, bias, sigmoid, groups=4, keep=2)
                assert np.array_equal(ids.cpu().numpy()[some], want)
                weights_match(w.cpu().numpy()[some], ww)
