"""A decoder layer's steps between its projections, written out in FP64: norm
and gate into INT8 rows, rotary positions, the 4-bit cache, attention over it.
Shares no code with the GPU path."""
import numpy as np

from . import aq_oracle as O


def norm(X, W, R=None, eps=1e-6, rounded=None):
    """(h, y): h = X + R rounded by `rounded` (FP32 -> FP32 of the rows' type), y the
    normed rows in FP32."""
    h = np.asarray(X, dtype=np.float32)
    if R is not None:
        h = h + np.asarray(R, dtype=np.float32)
        h = h if rounded is None else rounded(h)
    x = h.astype(np.float64)
    with np.errstate(all="ignore"):
        n = 1 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)
        return h, (x * n * np.asarray(W, dtype=np.float64)).astype(np.float32)


def swiglu(GU):
    """FP32 silu(gate) * up."""
    g, u = np.split(np.asarray(GU, dtype=np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        return (g / (1 + np.exp(-g)) * u).astype(np.float32)


def quant(Y):
    """aq_quant_act's codes and scales."""
    return O.quant_act(Y)


def rope(x, pos, freq, parts, interleaved=False):
    """x [M, heads, D] turned: FP64, rounded once to FP32."""
    x = np.array(x, dtype=np.float64)
    pos, freq, pairs = np.asarray(pos, dtype=np.float64), np.asarray(freq, dtype=np.float64), sum(parts)
    i = 0
    for axis, n in enumerate(parts):
        for _ in range(n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
            t = (pos[axis] * freq[i])[:, None]
            u, v = x[..., a].copy(), x[..., b].copy()
            x[..., a], x[..., b] = u * np.cos(t) - v * np.sin(t), v * np.cos(t) + u * np.sin(t)
            i += 1
    return x.astype(np.float32)


def hold(x):
    """(codes [..., D] of 0 .. 15, words uint32 [...]) of FP32 vectors."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    hi, lo = np.maximum(x.max(-1), 0), np.minimum(x.min(-1), 0)
    want = np.maximum((hi - lo) / 15, 1e-12)
    s = want.astype(np.float32)
    s = np.where(s.astype(np.float64) < want, np.nextafter(s, np.float32(np.inf)), s)
    bits = (s.view(np.uint32) + np.uint32(15)) & ~np.uint32(15)
    s = bits.view(np.float32).astype(np.float64)
    bad |= s >= 2.0 ** 64
    z = np.rint(-lo / s)
    c = np.clip(np.rint(x / s[..., None]) + z[..., None], 0, 15).astype(np.uint8)
    return np.where(bad[..., None], 0, c).astype(np.uint8), np.where(bad, np.uint32(0x7FC00000), bits | z.astype(np.uint32))


def packed(codes):
    """[..., D] codes as [..., D/2] bytes."""
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)


def values(bytes_, words):
    """What the cache's bytes [..., D/2] and words [...] stand for, FP64."""
    w = np.asarray(words).astype(np.uint32) if np.asarray(words).dtype != np.int32 else np.asarray(words).view(np.uint32)
    s = np.where(w < 0x5F800000, w & ~np.uint32(15), np.uint32(0x7FC00000)).astype(np.uint32).view(np.float32).astype(np.float64)
    c = np.stack([bytes_ & 15, bytes_ >> 4], -1).reshape(*bytes_.shape[:-1], 2 * bytes_.shape[-1]).astype(np.float64)
    return s[..., None] * (c - (w & 15)[..., None])


def attention(q, codes, words, table, kv_len, cu=None, scale=None, sums=None):
    """[M, Hq * D] in FP64, NaN rows where no sequence owns them; `sums` collects for
    each owned row and head (sum of weights times |v|, the sums |q||k| * scale, keys, the largest
    weight times a value's step, the largest score and exponent of a step in powers of two)."""
    q = np.asarray(q, dtype=np.float64)
    M, Hq, D = q.shape
    pages, _, heads, P, _ = codes.shape
    B, width = table.shape
    G, scale = Hq // heads, D ** -0.5 if scale is None else scale
    cu = np.arange(B + 1) if cu is None else np.asarray(cu)
    out = np.full((M, Hq, D), np.nan)
    for b in range(B):
        n, length = int(cu[b + 1] - cu[b]), int(np.clip(kv_len[b], 0, width * P))
        at = np.arange(length)
        page = table[b, at // P].astype(np.int64)
        there = (page >= 0) & (page < pages)
        at, page = at[there], page[there]
        for h in range(heads):
            k = values(codes[page, 0, h, at % P], words[page, 0, h, at % P])
            v = values(codes[page, 1, h, at % P], words[page, 1, h, at % P])
            for i in range(n):
                seen = at <= length - n + i
                m, ks, vs = int(cu[b]) + i, k[seen], v[seen]
                for j in range(h * G, h * G + G):
                    if not seen.any():
                        out[m, j] = 0
                        continue
                    with np.errstate(all="ignore"):
                        s = ks @ q[m, j] * scale
                        w = np.exp(s - s.max())
                        w /= w.sum()
                    out[m, j] = w @ vs
                    if sums is not None:
                        step = words[page, 1, h, at % P][seen] & np.uint32(0xFFFFFFF0)
                        step = np.maximum(step.view(np.float32).astype(np.float64), 2.0 ** -48)
                        sums[m, j] = (w @ np.abs(vs), np.abs(ks) @ np.abs(q[m, j]) * scale, int(seen.sum()),
                                      float((w * step).max()), float((np.abs(s) / np.log(2) + np.abs(np.log2(step))).max()))
    return out.reshape(M, Hq * D)
