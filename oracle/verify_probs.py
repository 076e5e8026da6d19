"""Verification of drafted tokens from probabilities (oracle; test-only).

The rule of verify.py with the distributions given instead of computed: p_i
and q_i are read as they are, an entry that is not a positive finite number
counts as 0, a block may be shorter than the row that holds it, and where the
row the next token is drawn from has no positive entry there is no token (-1).
Everything in float64."""

import numpy as np


def clean(row):
    row = np.asarray(row, dtype=np.float64)
    return np.where(np.isfinite(row) & (row > 0), row, 0.0)


def verify_block(p, q, tokens, u, length):
    """p [L+1, V], q [L, V], tokens [L], u [L+1], the block's length ->
    (n accepted, next token)."""
    L, V = len(tokens), np.shape(p)[1]
    length = min(max(int(length), 0), L)
    n = 0
    while n < length:
        d = int(tokens[n])
        if not 0 <= d < V:
            break
        pd, qd = clean(p[n][d:d + 1])[0], clean(q[n][d:d + 1])[0]
        if not float(u[n]) * qd < pd:
            break
        n += 1
    w = clean(p[n])
    if n < length:
        r = np.maximum(w - clean(q[n]), 0.0)
        if r.sum() > 0.0:
            w = r
    c = np.cumsum(w)
    if not c[-1] > 0.0:
        return n, -1
    goal = float(u[L]) * c[-1]
    return n, int(np.searchsorted(c, goal, side="right"))


def verify(p, q, tokens, u, lengths=None):
    """Batched -> (accept_len int32 [B], next_token int32 [B])."""
    B, L = np.shape(tokens)
    lengths = [L] * B if lengths is None else lengths
    got = [verify_block(p[b], q[b], tokens[b], u[b], lengths[b]) for b in range(B)]
    return (np.array([g[0] for g in got], np.int32).reshape(B),
            np.array([g[1] for g in got], np.int32).reshape(B))
