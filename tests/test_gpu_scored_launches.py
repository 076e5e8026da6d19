"""Which calls of routing and grouping by scores are one launch: up to 16 tokens, where
no lane of a wave holds more than eight experts."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say
from _launches import kernel_names

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def lane_experts(E, groups):
    """A group has the largest power of two of lanes that 64 leave it."""
    lanes = 1
    while groups * lanes * 2 <= 64:
        lanes *= 2
    return -(-(E // groups) // lanes)


@pytest.mark.parametrize("T,E,groups,one", [(1, 8, 1, True), (16, 256, 1, True), (16, 255, 17, True), (16, 384, 1, True),
                                            (16, 384, 48, True), (16, 512, 1, True), (16, 513, 1, False), (16, 297, 9, False),
                                            (1, 1024, 1, False), (17, 8, 1, False)])
def test_one_launch(mm, T, E, groups, one):
    say("launches of route_scored_permute", T, E, groups)
    assert one == (T <= 16 and lane_experts(E, groups) <= 8)
    logits = torch.from_numpy(np.random.default_rng(E).normal(size=(T, E)).astype(np.float32)).to(DEV)
    k = 4
    out = [torch.empty(s, dtype=d, device=DEV) for s, d in (((T, k), torch.int32), ((T, k), torch.float32), (E, torch.int32),
                                                            (E + 1, torch.int32), (T * k, torch.int32), (T * k, torch.int32))]
    names = ("topk_ids", "topk_w", "counts", "offsets", "sorted_pairs", "pair_to_row")
    found = kernel_names(lambda: mm.moe_route_scored_permute(logits, k, groups=groups, topk_groups=groups,
                                                             **dict(zip(names, out))))
    assert len(found) == (1 if one else 2), found


def test_every_size_up_to_256_experts():
    """What the header says of sizes: every E up to 256, and 384 in any number of groups."""
    for E in list(range(1, 257)) + [384]:
        for groups in range(1, min(64, E) + 1):
            assert E % groups or lane_experts(E, groups) <= 8
