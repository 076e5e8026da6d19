"""Refusals of routing by scores, of the layer that routes so and of low-rank
adapters: host checks only, nothing is enqueued."""

import math

import pytest
import torch

import mxfp4_moe_expert_route_amd as mm

P = 256        # an aligned fake device address: never dereferenced on error paths
SIGMOID, SOFTMAX = 1, 0


@pytest.fixture(scope="module")
def lib():
    return mm._lib.lib()


def bad_rules():
    """(T, E, k, score, groups, topk_groups, group_best, renormalise, scale), status"""
    ok = dict(T=8, E=384, k=8, score=SIGMOID, groups=8, keep=4, best=2, norm=1, scale=2.5)
    cases = [(dict(score=2), -3), (dict(score=-1), -3), (dict(T=-1), -2), (dict(E=0), -2), (dict(E=1032), -2),
             (dict(k=0), -2), (dict(k=33), -2), (dict(groups=0), -2), (dict(groups=5), -2), (dict(groups=96), -2),
             (dict(keep=0), -2), (dict(keep=9), -2), (dict(best=0), -2), (dict(best=3), -2),
             (dict(E=16, groups=8, keep=3, k=7), -2), (dict(E=4, groups=1, keep=1, k=5), -2),
             (dict(scale=math.inf), -2), (dict(scale=math.nan), -2), (dict(T=2 ** 31 - 1), -2)]
    for change, status in cases:
        r = {**ok, **change}
        yield tuple(r[n] for n in ("T", "E", "k", "score", "groups", "keep", "best", "norm", "scale")), status


RULE = (8, 384, 8, SIGMOID, 8, 4, 2, 1, 2.5)


def test_route_argument_checks(lib):
    f = lib.moe_route_scored
    for rule, status in bad_rules():
        assert f(P, P, *rule, P, P, None) == status, rule
    assert f(None, P, *RULE, P, P, None) == -1
    assert f(P, P, *RULE, None, P, None) == -1
    assert f(P, P, *RULE, P, None, None) == -1
    for i in range(4):
        a = [P, P, P, P]
        a[i] = P + 2
        assert f(a[0], a[1], *RULE, a[2], a[3], None) == -4
    assert f(None, None, 0, *RULE[1:], None, None, None) == 0


def test_route_permute_argument_checks(lib):
    f = lib.moe_route_scored_permute
    for rule, status in bad_rules():
        assert f(P, P, *rule, *[P] * 7, 1 << 30, None) == status, rule
    for i in [0] + list(range(2, 8)):
        a = [P] * 8
        a[i] = None
        assert f(a[0], a[1], *RULE, *a[2:], P, 0, None) == -1
    for i in range(8):
        a = [P] * 8
        a[i] = P + 1
        assert f(a[0], a[1], *RULE, *a[2:], P, 0, None) == -4
    big = (8192,) + RULE[1:]
    need = lib.moe_permute_workspace_bytes(8192, 384, 8)
    assert need > 0
    assert f(P, None, *big, *[P] * 7, need - 1, None) == -7
    assert f(P, None, *big, *[P] * 6, None, need, None) == -1
    assert f(P, None, *big, *[P] * 6, P + 2, need, None) == -4
    assert f(None, None, 0, *RULE[1:], *[None] * 7, 0, None) == 0


def test_layer_argument_checks(lib):
    f = lib.moe_mxfp4_scored_layer
    # x, logits, bias, T, H, I, E, k, score, groups, keep, best, norm, scale, 13 pointers, workspace, bytes, stream
    call = lambda T=8, H=6144, I=2048, rule=RULE, ptrs=None, ws=(P, 0): f(  # noqa: E731
        *(ptrs or [P] * 16)[:3], T, H, I, *rule[1:], *(ptrs or [P] * 16)[3:], *ws, None)
    for rule, status in bad_rules():
        assert call(T=rule[0], rule=rule, ws=(P, 1 << 30)) == status, rule
    for H, I in ((6160, 2048), (6144, 2040), (16416, 2048), (6144, 8224), (0, 32)):
        assert call(H=H, I=I) == -2
    for i in range(16):
        a = [P] * 16
        a[i] = None
        if i != 2:                                   # the bias may be NULL
            assert call(ptrs=a) == -1, i
        a[i] = P + 2
        assert call(ptrs=a) == -4, i
    assert call(T=8192, ws=(P, 64 * 384 * 4 - 1)) == -7
    assert call(T=8192, ws=(None, 64 * 384 * 4)) == -1
    assert call(T=0, ptrs=[None] * 16, ws=(None, 0)) == 0


def test_lora_argument_checks(lib):
    f = lib.lora_add         # x, rows, offsets, M, K, N, S, r, a, b, scale, y, dtype, ws, bytes, stream
    shape = (8, 64, 100, 4, 100)          # sizes that need a workspace
    need = lib.lora_add_workspace_bytes(*shape)
    assert need > 0
    ok = dict(p=[P] * 3, shape=shape, q=[P] * 4, dtype=1, ws=P, n=1 << 62)

    def call(**change):
        a = {**ok, **change}
        return f(*a["p"], *a["shape"], *a["q"], a["dtype"], a["ws"], a["n"], None)

    assert call(dtype=2) == -3
    for s in ((-1, 64, 100, 4, 16), ((1 << 20) + 1, 64, 100, 4, 16), (8, 0, 100, 4, 16), (8, 60, 100, 4, 16),
              (8, (1 << 17) + 8, 100, 4, 16), (8, 64, -1, 4, 16), (8, 64, (1 << 17) + 1, 4, 16), (8, 64, 100, 0, 16),
              (8, 64, 100, 1025, 16), (8, 64, 100, 4, 0), (8, 64, 100, 4, 129)):
        assert call(shape=s) == -2, s
        assert lib.lora_add_workspace_bytes(*s) == 0, s
    assert call(n=need - 1) == -7
    for i in range(3):
        p = [P] * 3
        p[i] = None
        assert call(p=p) == -1
    for i in (0, 1, 3):
        q = [P] * 4
        q[i] = None
        assert call(q=q) == -1
    assert call(ws=None) == -1
    for p in ([P + 8, P, P], [P, P + 2, P], [P, P, P + 2]):
        assert call(p=p) == -4
    for q in ([P + 8, P, P, P], [P, P + 8, P, P], [P, P, P + 2, P], [P, P, P, P + 1]):
        assert call(q=q) == -4
    assert call(q=[P, P, P, P + 2], dtype=0) == -4
    assert call(ws=P + 8) == -4
    assert call(shape=(0, 64, 100, 4, 16), p=[None] * 3, q=[None] * 4, ws=None, n=0) == 0
    assert call(shape=(8, 64, 0, 4, 16), p=[None] * 3, q=[None] * 4, ws=None, n=0) == 0
    assert lib.lora_add_workspace_bytes(0, 64, 100, 4, 16) == 0
    assert lib.lora_add_workspace_bytes(8, 64, 100, 4, 16) == 0          # one launch: none needed


def test_wrappers_refuse_host_tensors_and_wrong_types():
    logits = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mm.moe_route_scored(logits, 2)
    with pytest.raises(ValueError):
        mm.moe_route_scored(logits[0], 2)
    with pytest.raises(ValueError):
        mm.moe_route_scored(logits, 2, score="relu")
    with pytest.raises(TypeError):
        mm.moe_route_scored_permute(logits.double(), 2)
    with pytest.raises(ValueError):
        mm.moe_route_scored_permute(logits, 2)
    w = torch.zeros(8, 64, 16, dtype=torch.uint8)
    s = torch.zeros(8, 64, 1, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mm.moe_mxfp4_scored_layer(torch.zeros(4, 32, dtype=torch.bfloat16), logits, 2, w, s, w, s)
    x, i = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    a, b = torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.zeros(2, 5, 3, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mm.lora_add(x, i, i[:3], a, b, torch.zeros(4, 5))
    with pytest.raises(TypeError):
        mm.lora_add(x, i, i[:3], a, b, torch.zeros(4, 5).half())
    with pytest.raises(ValueError):
        mm.lora_add(x, i, i[:3], a[0], b, torch.zeros(4, 5))
