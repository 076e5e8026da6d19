"""The oracles of the MXFP4-activation products and of verification from
probabilities, pinned against brute force and closed forms."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import a4 as oa4
from oracle import layer as olayer
from oracle import mx as omx
from oracle import verify as ov
from oracle import verify_probs as ovp


def _mx(rng, rows, K, lo=120, hi=130):
    return (rng.integers(0, 256, (rows, K // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (rows, K // 32), dtype=np.uint8))


def _value(codes, scales, i):
    c = (int(codes[i // 2]) >> (4 * (i % 2))) & 15
    m, e = c & 1, (c >> 1) & 3
    mag = Fraction(m, 2) if e == 0 else (1 + Fraction(m, 2)) * Fraction(2) ** (e - 1)
    return (-mag if c & 8 else mag) * Fraction(2) ** (int(scales[i // 32]) - 127)


def test_gemm_against_exact_rationals():
    rng = np.random.default_rng(1)
    M, N, K = 3, 4, 96
    a, b = _mx(rng, M, K), _mx(rng, N, K)
    got, mag = oa4.gemm(*a, *b)
    for m in range(M):
        for n in range(N):
            terms = [_value(a[0][m], a[1][m], i) * _value(b[0][n], b[1][n], i) for i in range(K)]
            assert Fraction(float(got[m, n])) == sum(terms)
            assert Fraction(float(mag[m, n])) == sum(abs(t) for t in terms)


def test_contractions_are_the_layers_on_quantised_activations():
    """Against the bf16-activation oracle: MXFP4 values are bf16 values."""
    rng = np.random.default_rng(2)
    T, H, I, E, k = 5, 64, 32, 3, 2
    x = _mx(rng, T, H, 125, 129)
    w13 = [v.reshape(E, 2 * I, -1) for v in _mx(rng, E * 2 * I, H, 120, 124)]
    w2 = [v.reshape(E, H, -1) for v in _mx(rng, E * H, I, 120, 124)]
    logits = rng.standard_normal((T, E)).astype(np.float32)
    xb = omx.to_bf16_bits(omx.unpack(*x))
    ref = olayer.layer_forward(xb, logits, *w13, *w2, k)
    from oracle import permute as operm
    lists = operm.permute(ref["ids"], E)
    g, u, _, _ = oa4.gate_up(*x, lists["sorted_pairs"], lists["offsets"], k, *w13)
    h = omx.to_bf16_bits(oa4.silu(g) * u)
    p2r = lists["pair_to_row"].reshape(T, k)
    assert np.array_equal(h[p2r], ref["h_bits"])
    hq = omx.pack(omx.bf16_bits_to_f64(h))
    y, _ = oa4.down(*hq, lists["offsets"], *w2)
    for e in range(E):
        lo, hi = lists["offsets"][e], lists["offsets"][e + 1]
        np.testing.assert_array_equal(y[lo:hi], omx.unpack(hq[0][lo:hi], hq[1][lo:hi])
                                      @ omx.unpack(w2[0][e], w2[1][e]).T)


def test_verify_agrees_with_the_logit_form():
    rng = np.random.default_rng(3)
    B, L, V = 40, 4, 50
    logits = rng.normal(0, 2, (B, L + 1, V))
    p = np.stack([[ov.softmax64(r) for r in blk] for blk in logits])
    q = np.stack([[ov.softmax64(r + rng.normal(0, .5, V)) for r in blk[:L]] for blk in logits])
    tokens = np.array([[rng.choice(V, p=q[b, i]) for i in range(L)] for b in range(B)], np.int32)
    u = rng.random((B, L + 1))
    n, t = ovp.verify(p, q, tokens, u)
    for b in range(B):
        assert (n[b], t[b]) == ov.verify_block(logits[b], q[b], tokens[b], u[b])


@pytest.mark.parametrize("seed", range(3))
def test_verify_is_lossless(seed):
    """One drafted token, every (token, u_0, u_1) integrated: the output token
    is distributed as p_0."""
    rng = np.random.default_rng(seed)
    V, G = 5, 60
    p = rng.dirichlet(np.ones(V), 2)
    q = rng.dirichlet(np.ones(V), 1)
    grid = (np.arange(G) + 0.5) / G
    got = np.zeros(V)
    for d in range(V):
        for u0 in grid:
            n, _ = ovp.verify_block(p, q, [d], [u0, 0.5], 1)
            if n:
                got[d] += q[0, d] / G
            else:
                for u1 in grid:
                    got[ovp.verify_block(p, q, [d], [u0, u1], 1)[1]] += q[0, d] / G / G
    assert np.abs(got - p[0]).max() <= 0.02


def test_verify_edges():
    p = np.array([[0.0, 0.5, 0.5, 0.0], [0.25] * 4, [0.0, 0.0, 1.0, 0.0]])
    q = np.array([[0.0, 0.5, 0.5, 0.0], [0.25] * 4])
    # a drafter equal to the target is accepted for every u < 1
    assert ovp.verify_block(p, q, [1, 3], [0.999, 0.999, 0.0], 2) == (2, 2)
    # shorter block: drawn from the row after its end
    assert ovp.verify_block(p, q, [1, 3], [0.0, 0.0, 0.5], 1) == (1, 2)
    assert ovp.verify_block(p, q, [1, 3], [0.0, 0.0, 0.49], 0) == (0, 1)
    # no residual: from p itself; u = 0 takes the first token with probability
    assert ovp.verify_block(p, q, [0, 0], [0.0, 0.0, 0.0], 2) == (0, 1)
    # a token outside the vocabulary, rows without probability, bad entries
    assert ovp.verify_block(p, q, [4, 0], [0.0, 0.0, 0.9], 2) == (0, 2)
    assert ovp.verify_block(np.zeros((3, 4)), q, [1, 1], [0.0, 0.0, 0.3], 2) == (0, -1)
    bad = np.array([[np.nan, -1.0, np.inf, 0.5]] * 3)
    assert ovp.verify_block(bad, q, [2, 2], [0.0, 0.0, 0.0], 2) == (0, 3)
