"""CPU oracle for the gated block's training form -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may use it; it shares no code with the HIP library.  Everything
is float64 and follows the formulas of ``include/mgemm.h``; weights are given as
K x N whatever their storage.
"""
from __future__ import annotations

import numpy as np


def sigmoid(g):
    # exp of a non-positive number only: no overflow at either end.
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def forward(x, wg, wu):
    """(Z, G, U) of X (M x K) and the weights (K x N)."""
    g, u = x @ wg, x @ wu
    return g * sigmoid(g) * u, g, u


def pointwise(g, u, dz):
    """(dG, dU): the gradients at G and U."""
    s = sigmoid(g)
    return dz * u * s * (1.0 + g * (1.0 - s)), dz * g * s


def backward(x, wg, wu, g, u, dz):
    """(dX, dWg, dWu)."""
    dg, du = pointwise(g, u, dz)
    return dg @ wg.T + du @ wu.T, x.T @ dg, x.T @ du
