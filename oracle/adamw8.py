"""fp64 AdamW with moments in 8 bits: the update from the values that codes and scales stand for, and the values that the
new moments round to. Test infrastructure only."""
from __future__ import annotations

import numpy as np

BLOCK = 256
TOP = 448.0            # the largest e4m3 value
LEAST = 2.0 ** -9      # the smallest above zero
FLOOR = 2.0 ** -100


def nearest_code(y):
    """The e4m3 value nearest to y, ties to the even fraction: steps of 2^(e - 3) for 2^e <= |y| < 2^(e + 1), of 2^-9 at least."""
    y = np.asarray(y, np.float64)
    e = np.maximum(np.frexp(y)[1] - 4, -9)
    return np.clip(np.ldexp(np.round(np.ldexp(y, -e)), e), -TOP, TOP)


def quantise(x, root=False, still=None):
    """(codes, scales) of moments x (roots of second moments if root), blocks of BLOCK values, the last one short. still: where
    a first moment has no gradient; in a block where another has one, its codes below 2^-6 are rounded toward zero."""
    codes, scales = np.zeros_like(x), []
    for a in range(0, len(x), BLOCK):
        b = x[a:a + BLOCK]
        fine = np.isfinite(b)
        top = max(np.abs(b[fine]).max(initial=0.0), FLOOR)
        y = b * (TOP / top)
        if root:
            y = np.where(b > 0, np.maximum(y, LEAST), y)
        if still is not None and not still[a:a + BLOCK].all():
            y = np.where(still[a:a + BLOCK] & (np.abs(y) < 2.0 ** -6), np.trunc(y / LEAST) * LEAST, y)
        codes[a:a + BLOCK] = np.where(fine, nearest_code(np.where(fine, y, 0.0)), np.nan)
        scales.append(top / TOP)
    return codes, np.array(scales)


def spread(scales, n):
    return np.repeat(scales, BLOCK)[:n]


def update(p, g, m0, r0, step, *, lr, beta1, beta2, eps, weight_decay, l2=False):
    """From weights, gradients, first moments and roots of second moments (the values held) to the new ones, unrounded."""
    if l2:
        g, keep = g + weight_decay * p, 1.0
    else:
        keep = 1.0 - lr * weight_decay
    m = beta1 * m0 + (1.0 - beta1) * g
    r = np.sqrt(beta2 * r0 ** 2 + (1.0 - beta2) * g ** 2)
    with np.errstate(invalid="ignore", divide="ignore"):
        p = keep * p - lr * (m / (1.0 - beta1 ** step)) / (r / np.sqrt(1.0 - beta2 ** step) + eps)
    return p, m, r
