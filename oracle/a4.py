"""Products of two MXFP4 factors and the expert contractions on MXFP4
activations, by their definition in float64 (oracle; test-only).

The pages store the experts in MXFP4 and keep activations in higher precision
("MiMo-V2.5-Pro-FP4-DFlash" model card, §2 "FP4 Quantization"); MXFP4
activations are an addition, quantised by the same OCP conversion (mx.pack).
Every element is dequantised exactly and every sum is float64."""

import numpy as np

from . import mx


def gemm(a_codes, a_scales, b_codes, b_scales):
    """(a b^T [M, N], sum of the products' magnitudes [M, N]), float64."""
    a, b = mx.unpack(a_codes, a_scales), mx.unpack(b_codes, b_scales)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def silu(g):
    return g / (1.0 + np.exp(-g))


def gate_up(x_codes, x_scales, sorted_pairs, offsets, k, w13_codes, w13_scales):
    """(g, u, mag_g, mag_u) [rows, I] float64 for rows 0..offsets[E]-1; h is silu(g) u."""
    x = mx.unpack(x_codes, x_scales)
    E, I = w13_codes.shape[0], w13_codes.shape[1] // 2
    n = int(offsets[E])
    out = [np.zeros((n, I)) for _ in range(4)]
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi == lo:
            continue
        w = mx.unpack(w13_codes[e], w13_scales[e])
        xe = x[np.asarray(sorted_pairs[lo:hi]) // k]
        for half in range(2):
            out[half][lo:hi] = xe @ w[half * I:(half + 1) * I].T
            out[2 + half][lo:hi] = np.abs(xe) @ np.abs(w[half * I:(half + 1) * I]).T
    return tuple(out)


def down(h_codes, h_scales, offsets, w2_codes, w2_scales):
    """(y, magnitudes) [rows, H] float64 for rows 0..offsets[E]-1."""
    E, H = w2_codes.shape[:2]
    n = int(offsets[E])
    h = mx.unpack(h_codes, h_scales)
    y, mag = np.zeros((n, H)), np.zeros((n, H))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            w = mx.unpack(w2_codes[e], w2_scales[e])
            y[lo:hi] = h[lo:hi] @ w.T
            mag[lo:hi] = np.abs(h[lo:hi]) @ np.abs(w).T
    return y, mag
