"""Attention over packed sequences in NumPy, 64 bits throughout [klein, section 4.3, with segments, visible keys, capped
scores and a distance bias]."""

import numpy as np


def attention_packed(q, k, v, q_start, k_start, visible=None, scale=1.0, cap=0.0, slope=None):
    """q [rows, heads, d], k, v [keys, kv_heads, d] -> o, lse [heads, rows], and sum_j w_ij |v_j| / sum_j w_ij (what a
    rounding of the weights is measured by). Rows of no segment: NaN."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    rows, heads, d = q.shape
    o, mag, lse = np.full((rows, heads, d), np.nan), np.full((rows, heads, d), np.nan), np.full((heads, rows), np.nan)
    for s in range(len(q_start) - 1):
        q0, q1, k0, k1 = q_start[s], q_start[s + 1], k_start[s], k_start[s + 1]
        nq, nk = q1 - q0, k1 - k0
        for h in range(heads):
            g = h * k.shape[1] // heads
            for i in range(nq):
                n = nk if visible is None else min(max(int(visible[q0 + i]), 0), nk)
                if n == 0:
                    o[q0 + i, h], mag[q0 + i, h], lse[h, q0 + i] = 0.0, 0.0, -np.inf
                    continue
                x = k[k0:k0 + n, g] @ q[q0 + i, h] * scale
                if cap:
                    x = cap * np.tanh(x / cap)
                if slope is not None:
                    x = x - slope[h] * np.abs(i + nk - nq - np.arange(n))
                m = x.max()
                w = np.exp(x - m)
                lse[h, q0 + i] = m + np.log(w.sum())
                o[q0 + i, h] = w @ v[k0:k0 + n, g] / w.sum()
                mag[q0 + i, h] = w @ np.abs(v[k0:k0 + n, g]) / w.sum()
    return o, lse, mag
