"""Oracle for the gated linear recurrence (TEST INFRASTRUCTURE: only tests/
may use it).

Plain float64 numpy, row by row:
  h_t = a_t h_{t-1} + u_t, u_t = x_t, or (1 - a_t) x_t when coupled (the
  compositing recurrence of "Gaussian Splatting反向传播的CUDA实现", section 2,
  with gate 1 - alpha),
and the chain rule through it.  ``forward`` also returns the recurrence of the
magnitudes |a|, |u|, |h0|, which bounds the rounding error of any order of
evaluation.  Parity pinned by tests/test_oracle_scan.py.
"""
from __future__ import annotations

import numpy as np


def _rows(beg, end, reverse):
    return range(end - 1, beg - 1, -1) if reverse else range(beg, end)


def _wide(a, C):
    return np.repeat(np.asarray(a, np.float64), C // a.shape[1], axis=1)


def forward(a, x, offsets, h0=None, reverse=False, coupled=False, magnitude=False):
    """a [T, G], x [T, C], offsets [S + 1], h0 [S, C] or None.  Returns (h
    [T, C], h_last [S, C], before [T, C]: the state in front of each row);
    rows of no sequence are 0.  With ``magnitude`` every factor and term is
    replaced by its absolute value ((1 - a) x by |1 - a| |x|)."""
    x = np.asarray(x, np.float64)
    T, C = x.shape
    A = _wide(a, C)
    u = (1.0 - A) * x if coupled else x.copy()
    S = len(offsets) - 1
    s0 = np.zeros((S, C)) if h0 is None else np.asarray(h0, np.float64)
    if magnitude:
        A, u, s0 = np.abs(A), np.abs(u), np.abs(s0)
    h, before = np.zeros((T, C)), np.zeros((T, C))
    last = s0.copy()
    for s in range(S):
        state = s0[s].copy()
        for t in _rows(offsets[s], offsets[s + 1], reverse):
            before[t] = state
            state = A[t] * state + u[t]
            h[t] = state
        last[s] = state
    return h, last, before


def backward(a, x, offsets, before, dh=None, dh_last=None, reverse=False, coupled=False, magnitude=False):
    """Gradients (da [T, G], dx [T, C], dh0 [S, C]) given ``before`` of
    forward (of the same ``magnitude``)."""
    x = np.asarray(x, np.float64)
    T, C = x.shape
    G = a.shape[1]
    A = _wide(a, C)
    S = len(offsets) - 1
    up = np.zeros((T, C)) if dh is None else np.asarray(dh, np.float64)
    k = np.zeros((S, C)) if dh_last is None else np.asarray(dh_last, np.float64).copy()
    one_minus, val = 1.0 - A, (before - x if coupled else before)
    if magnitude:
        A, up, k, one_minus = np.abs(A), np.abs(up), np.abs(k), np.abs(one_minus)
        val = before + np.abs(x) if coupled else before
    da, dx = np.zeros((T, G)), np.zeros((T, C))
    for s in range(S):
        for t in list(_rows(offsets[s], offsets[s + 1], reverse))[::-1]:
            g = up[t] + k[s]
            da[t] = (g * val[t]).reshape(G, C // G).sum(1)
            dx[t] = one_minus[t] * g if coupled else g
            k[s] = A[t] * g
    return da, dx, k
