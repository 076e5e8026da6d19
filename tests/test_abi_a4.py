"""Refusals of the MXFP4-activation entry points and of verification from
probabilities: host checks only, nothing is enqueued."""

import pytest
import torch

import mxfp4_moe_expert_route_amd as mm

P = 256        # an aligned fake device address: never dereferenced on error paths


@pytest.fixture(scope="module")
def lib():
    return mm._lib.lib()


def test_gemm_argument_checks(lib):
    f = lib.mxfp4_gemm       # a, as, b, bs, M, N, K, c, dtype, stream
    assert f(P, P, P, P, 4, 8, 64, P, 2, None) == -3
    assert f(P, P, P, P, 4, 8, 48, P, 0, None) == -2
    assert f(P, P, P, P, 4, 8, 0, P, 0, None) == -2
    assert f(P, P, P, P, 4, 8, (1 << 20) + 32, P, 0, None) == -2
    assert f(P, P, P, P, -1, 8, 64, P, 0, None) == -2
    assert f(P, P, P, P, (1 << 30) + 1, 8, 32, P, 0, None) == -2
    assert f(P, P, P, P, 8, (1 << 30) + 1, 32, P, 0, None) == -2
    assert f(P, P, P, P, 4, -8, 64, P, 0, None) == -2
    for i in range(4):
        a = [P] * 4
        a[i] = None
        assert f(*a, 4, 8, 64, P, 0, None) == -1
    assert f(P, P, P, P, 4, 8, 64, None, 0, None) == -1
    assert f(P + 8, P, P, P, 4, 8, 64, P, 0, None) == -4
    assert f(P, P, P + 4, P, 4, 8, 64, P, 0, None) == -4
    assert f(P, P, P, P, 4, 8, 64, P + 2, 0, None) == -4
    assert f(P, P, P, P, 4, 8, 64, P + 1, 1, None) == -4
    assert f(None, None, None, None, 0, 8, 64, None, 0, None) == 0
    assert f(None, None, None, None, 4, 0, 64, None, 1, None) == 0


def test_gate_up_argument_checks(lib):
    f = lib.moe_mxfp4_a4_gate_up_swiglu
    # xc, xs, pairs, offsets, T, H, I, E, k, wc, ws, h, hc, hs, stream
    assert f(P, P, P, P, 8, 6160, 2048, 384, 8, P, P, P, None, None, None) == -2
    assert f(P, P, P, P, 8, 6144, 2040, 384, 8, P, P, P, None, None, None) == -2
    assert f(P, P, P, P, 8, 16416, 2048, 384, 8, P, P, P, None, None, None) == -2
    assert f(P, P, P, P, 8, 6144, 2048, 1025, 8, P, P, P, None, None, None) == -2
    assert f(P, P, P, P, 8, 6144, 2048, 4, 5, P, P, P, None, None, None) == -2
    assert f(P, P, P, P, 1 << 30, 32, 32, 4, 4, P, P, P, None, None, None) == -2
    assert f(P, P, None, P, 8, 6144, 2048, 384, 8, P, P, P, None, None, None) == -1
    # exactly one form of h
    assert f(P, P, P, P, 8, 6144, 2048, 384, 8, P, P, None, None, None, None) == -1
    assert f(P, P, P, P, 8, 6144, 2048, 384, 8, P, P, None, P, None, None) == -1
    assert f(P, P, P, P, 8, 6144, 2048, 384, 8, P, P, P, P, P, None) == -1
    assert f(P + 8, P, P, P, 8, 6144, 2048, 384, 8, P, P, P, None, None, None) == -4
    assert f(P, P, P, P, 8, 6144, 2048, 384, 8, P, P, None, P + 8, P, None) == -4
    assert f(P, P, P, P + 2, 8, 6144, 2048, 384, 8, P, P, P, None, None, None) == -4
    assert f(None, None, None, None, 0, 6144, 2048, 384, 8, None, None, None, None, None, None) == 0


def test_down_argument_checks(lib):
    f = lib.moe_mxfp4_a4_down       # hc, hs, offsets, T, H, I, E, k, wc, ws, y, stream
    assert f(P, P, P, 8, 6144, 2064, 384, 8, P, P, P, None) == -2
    assert f(P, P, P, 8, 6144, 8224, 384, 8, P, P, P, None) == -2
    assert f(P, P, P, 8, 6144, 2048, 384, 33, P, P, P, None) == -2
    assert f(P, P, P, 8, 6144, 2048, 384, 8, P, P, None, None) == -1
    assert f(P, P, P, 8, 6144, 2048, 384, 8, P, P, P + 4, None) == -4
    assert f(P, P, P, 8, 6144, 2048, 384, 8, P + 8, P, P, None) == -4
    assert f(None, None, None, 0, 6144, 2048, 384, 8, None, None, None, None) == 0


def test_layer_argument_checks(lib):
    f = lib.moe_mxfp4_a4_layer
    shape = (8, 6144, 2048, 384, 8)
    for i in range(18):
        a = [P] * 18
        a[i] = None
        assert f(a[0], a[1], *shape, *a[2:], P, 0, None) == -1, i
    assert f(P, P, 8192, 6144, 2048, 384, 8, *[P] * 16, P, 64 * 384 * 4 - 1, None) == -7
    assert f(P, P, 8192, 6144, 2048, 384, 8, *[P] * 16, None, 64 * 384 * 4, None) == -1
    assert f(P, P, 8, 6144, 2048, 4, 8, *[P] * 16, P, 0, None) == -2
    assert f(P + 8, P, *shape, *[P] * 16, P, 0, None) == -4
    assert f(P, P, 0, 6144, 2048, 384, 8, *[None] * 16, None, 0, None) == 0


def test_verify_probs_argument_checks(lib):
    f = lib.dflash_verify_probs
    # p, q, dtype, tokens, len, u, B, L, V, accept, next, ws, bytes, stream
    V = 50000
    ws = lib.dflash_verify_probs_workspace_bytes(4, 8, V)
    assert ws > 0
    assert lib.dflash_verify_probs_workspace_bytes(4, 8, 50) == 0      # one launch: none needed
    assert lib.dflash_verify_probs_workspace_bytes(4, 33, 50) == 0
    assert lib.dflash_verify_probs_workspace_bytes(4, 8, 0) == 0
    assert lib.dflash_verify_probs_workspace_bytes(0, 8, 50) == 0
    assert f(P, P, 5, P, None, P, 4, 8, V, P, P, P, ws, None) == -3
    assert f(P, P, 0, P, None, P, 4, 0, V, P, P, P, ws, None) == -2
    assert f(P, P, 0, P, None, P, 4, 33, V, P, P, P, ws, None) == -2
    assert f(P, P, 0, P, None, P, 4, 8, 0, P, P, P, ws, None) == -2
    assert f(P, P, 0, P, None, P, (1 << 24) + 1, 8, V, P, P, P, 1 << 40, None) == -2
    assert f(P, P, 0, P, None, P, (1 << 20) + 1, 1, 3, P, P, P, 0, None) == -2
    assert f(P, P, 0, P, None, P, 4, 8, V, P, P, P, ws - 1, None) == -7
    assert f(P, None, 0, P, None, P, 4, 8, V, P, P, P, ws, None) == -1
    assert f(P, P, 0, P, None, P, 4, 8, V, P, P, None, ws, None) == -1
    assert f(P + 2, P, 0, P, None, P, 4, 8, V, P, P, P, ws, None) == -4
    assert f(P, P + 1, 1, P, None, P, 4, 8, V, P, P, P, ws, None) == -4
    assert f(P, P, 1, P, P + 2, P, 4, 8, V, P, P, P, ws, None) == -4
    assert f(P, P, 1, P, None, P, 4, 8, V, P, P, P + 4, ws, None) == -4
    assert f(None, None, 0, None, None, None, 0, 8, 50, None, None, None, 0, None) == 0


def test_wrappers_refuse_host_tensors_and_wrong_ranks():
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mm.mxfp4_gemm(c, s, c, s)
    with pytest.raises(ValueError):
        mm.mxfp4_gemm(c[0], s[0], c, s)
    with pytest.raises(TypeError):
        mm.mxfp4_gemm(c, s, c, s, dtype=torch.float16)
    i32 = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        mm.moe_mxfp4_a4_gate_up_swiglu(c, s, i32, i32, 2, c, s)
    with pytest.raises(ValueError):
        mm.moe_mxfp4_a4_down(c, s, i32, 3, c[None], s[None])
    with pytest.raises(ValueError):
        mm.dflash_verify_probs(torch.zeros(1, 3, 8), torch.zeros(1, 2, 8), i32, i32)
    with pytest.raises(TypeError):
        mm.dflash_verify_probs(torch.zeros(1, 3, 8).half(), torch.zeros(1, 2, 8).half(), i32, i32)


def test_verify_probs_workspace_of_refused_sizes(lib):
    f = lib.dflash_verify_probs_workspace_bytes
    most_b, most_v = 1 << 20, 1 << 30
    assert f(1, 1, most_v) > 0 and f(1, 32, most_v) > 0 and f(most_b, 1, 8193) > 0
    for B, L, V in ((most_b + 1, 1, 8193), (most_b + 1, 1, 3), (2 ** 31 - 1, 1, 50000), (-1, 1, 50000),
                    (1, 1, most_v + 1), (1, 1, 2 ** 31 - 1), (1, 33, 50000), (1, 0, 50000)):
        assert f(B, L, V) == 0, (B, L, V)
        assert lib.dflash_verify_probs(P, P, 0, P, None, P, B, L, V, P, P, P, 1 << 40, None) == -2
