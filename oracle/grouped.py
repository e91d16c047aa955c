"""Plain 64-bit forms of the products grouped by an index: plans, router, experts, combine, adapters.

Inputs are numpy arrays (bf16 as uint16 bit patterns); every sum is taken in fp64.
"""
from __future__ import annotations

import numpy as np

from oracle import benq


def group_rows(index: np.ndarray, groups: int):
    """order [M] (rows of group 0 ascending, then group 1, ...; -1 past the last), offsets [groups + 1]."""
    lists = [[i for i, g in enumerate(index) if g == want] for want in range(groups)]
    flat = [i for rows in lists for i in rows]
    offsets = np.cumsum([0] + [len(rows) for rows in lists])
    return np.array(flat + [-1] * (len(index) - len(flat)), dtype=np.int32), offsets.astype(np.int32)


def route(logits: np.ndarray, k: int, normalize: bool):
    """experts [T, k] and weights [T, k] (fp64) of logits [T, E] (finite or -inf)."""
    T, E = logits.shape
    experts = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = [e for e in range(E) if l[e] != -np.inf]
        chosen = sorted(live, key=lambda e: (-l[e], e))[:k]
        if not chosen:
            continue
        p = {e: np.exp(l[e] - l[chosen[0]]) for e in live}
        total = sum(p[e] for e in (chosen if normalize else live))
        for j, e in enumerate(chosen):
            experts[t, j], weights[t, j] = e, p[e] / total
    return experts, weights


def grouped_linear(codes, lut, x_bits, offsets, xr, K):
    """Per position i of group g: (y, s) with y[i] = W_g x[xr[i]] and s[i] = |W_g| |x[xr[i]]|, fp64 [M, N]."""
    M, N = len(xr), codes.shape[1]
    y, s = np.zeros((M, N)), np.zeros((M, N))
    x = benq.bf16_to_f32(x_bits).astype(np.float64)
    for g in range(codes.shape[0]):
        rows = slice(int(offsets[g]), int(offsets[g + 1]))
        if rows.start >= rows.stop:
            continue
        W = benq.dequant(codes[g], lut[g], K).astype(np.float64)
        xs = x[np.asarray(xr[rows])]
        y[rows], s[rows] = xs @ W.T, np.abs(xs) @ np.abs(W).T
    return y, s


def combine(y, experts, weights, residual):
    """out [T, N] fp64 and the sum of the terms' magnitudes; y [T * k, N]."""
    T, k = experts.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if experts[t, j] >= 0:
                term = float(weights[t, j]) * y[t * k + j].astype(np.float64)
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def lora(A_bits, B_bits, y, x_bits, index, scale):
    """y + scale_g B_g (A_g x) for rows of adapter g = index (fp64 [T, N]), and |scale| |B| (|A| |x|)."""
    x = benq.bf16_to_f32(x_bits).astype(np.float64)
    out, mag = y.astype(np.float64).copy(), np.zeros(y.shape)
    for i, g in enumerate(index):
        if 0 <= g < A_bits.shape[0]:
            A = benq.bf16_to_f32(A_bits[g]).astype(np.float64)
            B = benq.bf16_to_f32(B_bits[g]).astype(np.float64)
            f = 1.0 if scale is None else float(scale[g])
            out[i] += f * (B @ (A @ x[i]))
            mag[i] = abs(f) * (np.abs(B) @ (np.abs(A) @ np.abs(x[i])))
    return out, mag
