"""Plain FP64 definitions of the per-token-factor operators: the router, the
experts' layer over quantized experts and the low-rank adapters.  Shares no
code with the HIP path."""

from __future__ import annotations

import numpy as np

from . import aq_oracle as O


def route(X, Wr, top_k, bias=None, score="softmax", norm=True, scale=1.0):
    """ids INT32 [M, top_k] (-1: no expert left) and FP64 weights."""
    X, Wr = np.asarray(X, dtype=np.float64), np.asarray(Wr, dtype=np.float64)
    l = X @ Wr.T
    if score == "softmax":
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        key = l.copy()
    else:
        p = 1 / (1 + np.exp(-l))
        key = p.copy()
    if bias is not None:
        key = key + np.asarray(bias, dtype=np.float64)[None, :]
    M, E = l.shape
    ids = np.full((M, top_k), -1, dtype=np.int32)
    w = np.zeros((M, top_k))
    for m in range(M):
        order = sorted(range(E), key=lambda e: (-key[m, e], e))
        chosen = [e for e in order[:top_k] if key[m, e] > -np.inf]
        ids[m, :len(chosen)] = chosen
        w[m, :len(chosen)] = p[m, chosen]
        if norm and chosen:
            if score == "softmax":     # the same ratio, without underflow of far logits
                q = np.exp(l[m, chosen] - l[m, chosen].max())
                w[m, :len(chosen)] = q
            total = w[m].sum()
            w[m] = w[m] / total if total > 0 else 0.0
    return ids, scale * w


def linear64(qx, sx, codes, sW, bK):
    """sx[m] sum_j sW[n, j] P[m, n, j] in FP64, and the sum of the magnitudes."""
    P = O.tile_partials(np.asarray(qx, dtype=np.int64), codes, bK).astype(np.float64)
    s = np.asarray(sx, dtype=np.float32).astype(np.float64)[:, None]
    terms = P * np.asarray(sW, dtype=np.float32).astype(np.float64)[None]
    return s * terms.sum(-1), np.abs(s) * np.abs(terms).sum(-1)


def experts(qx, sx, ids, weights, gate_up, down, E, bK=128):
    """Y FP64 [M, H] and the sum of magnitudes of its terms.  gate_up and down
    are (codes, sW) of the whole [E*2I, H] and [E*H, I] projections."""
    (c13, s13), (c2, s2) = gate_up, down
    H, I = c13.shape[1], c2.shape[1]
    ids = np.asarray(ids)
    M, k = ids.shape
    Y, mag = np.zeros((M, H)), np.zeros((M, H))
    for m in range(M):
        for i in range(k):
            e = int(ids[m, i])
            if not 0 <= e < E:
                continue
            gu, _ = linear64(qx[m:m + 1], sx[m:m + 1], c13[e * 2 * I:(e + 1) * 2 * I], s13[e * 2 * I:(e + 1) * 2 * I], bK[0] if isinstance(bK, tuple) else bK)
            g, u = gu[:, :I], gu[:, I:]
            with np.errstate(over="ignore"):
                h = (g / (1 + np.exp(-g)) * u).astype(np.float32)
            qh, sh = O.quant_act(h)
            y, a = linear64(qh, sh.astype(np.float32), c2[e * H:(e + 1) * H], s2[e * H:(e + 1) * H], bK[1] if isinstance(bK, tuple) else bK)
            w = float(np.float32(weights[m, i]))
            Y[m] += w * y[0]
            mag[m] += abs(w) * a[0]
    return Y, mag


def lora(Y, X, ids, A, B, scale=None, ranks=None):
    """Y FP64 [M, N] and the sum of magnitudes of its terms."""
    Y, X = np.asarray(Y, dtype=np.float64), np.asarray(X, dtype=np.float64)
    A, B = np.asarray(A, dtype=np.float64), np.asarray(B, dtype=np.float64)
    L, R, _ = A.shape
    out, mag = Y.copy(), np.abs(Y)
    for m, a in enumerate(np.asarray(ids)):
        if not 0 <= a < L:
            continue
        r = R if ranks is None else min(max(int(ranks[a]), 0), R)
        s = 1.0 if scale is None else float(scale[a])
        out[m] += s * (B[a, :, :r] @ (A[a, :r] @ X[m]))
        mag[m] += abs(s) * (np.abs(B[a, :, :r]) @ (np.abs(A[a, :r]) @ np.abs(X[m])))
    return out, mag
