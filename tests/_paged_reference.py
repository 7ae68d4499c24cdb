"""Plain fp64 loops of the paged serving operators (test infrastructure), one sequence, head
and row at a time, on numpy arrays."""
import math

import numpy as np


def rotate(x, pos, freq, interleaved, scale=1.0, back=False):
    """x [..., d] at one position."""
    y = np.array(x, np.float64)
    rot = 2 * len(freq)
    for i, f in enumerate(freq):
        a = math.fmod(float(pos) * float(f), 2 * math.pi)
        c, s = math.cos(a) * scale, math.sin(a) * scale
        s = -s if back else s
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        x1, x2 = y[..., p].copy(), y[..., q].copy()
        y[..., p], y[..., q] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def sigma(x):
    return np.where(x > 0, x + 1.0, np.exp(np.minimum(x, 0.0)))


def row_at(table_row, r, page, P):
    """(page, slot) of row r, or None outside the cache."""
    i = r // page
    if i >= len(table_row) or not 0 <= table_row[i] < P:
        return None
    return int(table_row[i]), r % page


def attend(q, rows_k, rows_v):
    """q [d], rows [n, d] -> (output, weights); zeros for no rows."""
    if len(rows_k) == 0:
        return np.zeros_like(q), np.zeros(0)
    x = rows_k @ q / math.sqrt(len(q))
    p = np.exp(x - x.max())
    p /= p.sum()
    return p @ rows_v, p


def select(w, budget, recent):
    """Rows kept of accumulated weights w [n], ascending."""
    n = len(w)
    if n <= budget:
        return list(range(n))
    old = n - min(recent, n)
    key = [(-math.inf if math.isnan(w[i]) else -w[i], i) for i in range(old)]
    key.sort()
    return sorted(i for _, i in key[:budget - (n - old)]) + list(range(old, n))
