"""Grouping of pairs whose tokens name one expert more than once, or all the same:
the lists are the stable ones, and such ids cost about what distinct ones do."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def ids_of(kind, rng, T, E, k):
    if kind == "distinct":
        return rng.random((T, E)).argsort(1)[:, :k].astype(np.int32)
    if kind == "token":                                   # a token names one expert k times
        return np.repeat(rng.integers(0, E, (T, 1)), k, axis=1).astype(np.int32)
    if kind == "column":                                  # all tokens name the same k
        return np.tile(rng.integers(0, E, k), (T, 1)).astype(np.int32)
    if kind == "halves":
        return np.where(np.arange(T * k).reshape(T, k) < T * k // 2, 0, E - 1).astype(np.int32)
    ids = np.full((T, k), E // 2, np.int32)               # "same"
    ids[::7, 0] = -1
    return ids


# both sides of 65536 + 128 E pairs and of 131072, and few experts
@pytest.mark.parametrize("T,E,k", [(16608, 7, 4), (16609, 7, 4), (14336, 384, 8), (14337, 384, 8), (32768, 1024, 4),
                                   (32769, 1024, 4), (2049, 4, 4), (3001, 5, 5), (300, 32, 32), (8500, 640, 8)])
def test_lists(mm, T, E, k):
    rng = np.random.default_rng([T, E, k])
    for kind in ("token", "column", "halves", "same"):
        say("permute repeats", T, E, k, kind)
        ids = ids_of(kind, rng, T, E, k)
        counts, offsets, pairs, row = (v.cpu().numpy() for v in mm.moe_permute(torch.from_numpy(ids).to(DEV), E))
        flat = ids.ravel()
        at = np.flatnonzero(flat >= 0)
        at = at[np.argsort(flat[at], kind="stable")]
        want = np.full(T * k, -1)
        want[at] = np.arange(len(at))
        assert np.array_equal(counts, np.bincount(flat[flat >= 0], minlength=E))
        assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(counts)]))
        assert np.array_equal(pairs[:len(at)], at) and np.array_equal(row, want)


def test_repeated_ids_cost_what_distinct_ones_do(mm):
    """64 lanes that meet on one counter once took five times as long here; the bound
    is twice, of the least of several timings each."""
    rng = np.random.default_rng(1)
    T, E, k, calls = 8192, 384, 8, 20
    graphs = {}
    for kind in ("distinct", "token", "column", "same"):
        ids = torch.from_numpy(ids_of(kind, rng, T, E, k)).to(DEV)
        out = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (E, E + 1, T * k, T * k)]
        ws = torch.empty(mm.moe_permute_workspace_bytes(T, E, k), dtype=torch.uint8, device=DEV)
        mm.moe_permute(ids, E, *out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(calls):
                mm.moe_permute(ids, E, *out, workspace=ws)
        graphs[kind] = (graph, ids, out, ws)
    least = dict.fromkeys(graphs, float("inf"))
    for _ in range(9):
        for kind, (graph, *_rest) in graphs.items():
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            least[kind] = min(least[kind], a.elapsed_time(b) * 1e3 / calls)
    say("permute", {kind: round(t, 1) for kind, t in least.items()}, "us")
    assert max(least.values()) <= 2 * least["distinct"]
