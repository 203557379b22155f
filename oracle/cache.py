"""Float64 forms of the paged-cache operators (norm + rotation + store,
attention of one new token, eviction by accumulated weight).

Written over contiguous sequences: pages are gathered by `sequence` and
compared with what the kernels left in theirs.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

F64 = np.float64


def head_norm(x, gain, eps):
    """x / sqrt(mean(x^2) + eps) * gain over each head; gain None = x."""
    x = np.asarray(x, F64)
    if gain is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(gain, F64)


def rotate(x, pos, theta):
    """Rotate-half rotation of [..., heads, hd] at positions [...]: the pairs
    (j, j + hd/2) as complex numbers times e^{i pos theta^(-2j/hd)}."""
    x = np.asarray(x, F64)
    half = x.shape[-1] // 2
    freq = float(theta) ** (-np.arange(half) / half)
    turn = np.exp(1j * np.asarray(pos, F64)[..., None] * freq)[..., None, :]
    z = (x[..., :half] + 1j * x[..., half:]) * turn
    return np.concatenate([z.real, z.imag], axis=-1)


def sequence(pages, table_row, n, page):
    """Rows 0..n-1 of a sequence gathered from its pages, one by one."""
    out = [pages[table_row[j // page], j % page] for j in range(n)]
    return np.stack(out) if out else np.zeros((0,) + pages.shape[2:], pages.dtype)


def attend_one(q, k, v, scale):
    """q [nq, hd], k and v [n, nkv, hd] -> out [nq, hd], weights [nq, n]."""
    q, k, v = (np.asarray(t, F64) for t in (q, k, v))
    nq, nkv = q.shape[0], k.shape[1]
    out, weights = np.zeros_like(q), np.zeros((nq, k.shape[0]))
    if k.shape[0] == 0:
        return out, weights
    for h in range(nq):
        c = h // (nq // nkv)
        s = k[:, c] @ q[h] * scale
        e = np.exp(s - s.max())
        weights[h] = e / e.sum()
        out[h] = weights[h] @ v[:, c]
    return out, weights


def choose(weights, n, budget, n_first, n_recent):
    """Kept positions (ascending) of one sequence and head, by repeated
    choice: NaN below every number, -0 equal to 0, ties to the lower index."""
    if n <= budget:
        return list(range(n))
    kept = set(range(n_first)) | set(range(n - n_recent, n))
    rest = [j for j in range(n) if j not in kept]
    rest.sort(key=lambda j: (1, 0.0, j) if np.isnan(weights[j]) else (0, -float(weights[j]) + 0.0, j))
    kept |= set(rest[:budget - n_first - n_recent])
    return sorted(kept)
