"""model.Decoder without a GPU: its calls answered by the FP64 oracle, so that what it joins to what shows."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import mixed_precision_int_amd.model as mdl
from oracle import layer as RL

H, I, HEADS, KV, D, LAYERS, P = 64, 128, 4, 2, 64, 3, 16
EPS = 1e-5
GEOMETRY = dict(qkv=((HEADS + 2 * KV) * D, H), o=(H, HEADS * D), gate_up=(2 * I, H), down=(H, I))


def packed(W):
    """Stands for a packed projection: its rows in FP64."""
    return SimpleNamespace(N=W.shape[0], K=W.shape[1], W=W, s8=torch.empty(0))


def cache_of(pages):
    return SimpleNamespace(codes=np.zeros((pages, 2, KV, P, D // 2), np.uint8), words=np.zeros((pages, 2, KV, P), np.uint32))


def rows_of(y):
    q, s = RL.quant(y)
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(s.astype(np.float32))


class Oracle:
    """The library's calls on host tensors, by the oracle."""

    @staticmethod
    def aq_norm_quant(X, weight, residual=None, eps=1e-6, h=None):
        hh, y = RL.norm(X.numpy(), weight.numpy(), None if residual is None else residual.numpy(), eps)
        if residual is None:
            return rows_of(y)
        h = torch.empty_like(X) if h is None else h
        h.copy_(torch.from_numpy(hh))
        return (*rows_of(y), h)

    @staticmethod
    def aq_quant_act(X, mark=False):
        assert mark
        return rows_of(X.numpy())

    @staticmethod
    def aq_swiglu_quant(gate_up):
        return rows_of(RL.swiglu(gate_up.numpy()))

    @staticmethod
    def aq_linear_decode(pw, qx, sx, out=None, **k):
        assert qx.shape[0] <= 64 and out is None
        return torch.from_numpy((sx.numpy()[:, None] * (qx.numpy().astype(np.float64) @ pw.W.T)).astype(np.float32))

    @staticmethod
    def aq_linear_prefill(pw, qx, sx, out=None, **k):
        assert qx.shape[0] > 64 and out is None
        return torch.from_numpy((sx.numpy()[:, None] * (qx.numpy().astype(np.float64) @ pw.W.T)).astype(np.float32))

    @staticmethod
    def aq_rope_kv4(qkv, rope, positions, cache, slots, out):
        x = qkv.numpy().reshape(qkv.shape[0], -1, D)
        t = x[:, :HEADS + KV] if rope is None else RL.rope(x[:, :HEADS + KV], positions.numpy()[None], rope.freq, rope.parts)
        c, w = RL.hold(np.stack([t[:, HEADS:], x[:, HEADS + KV:]], 1))
        for m, s in enumerate(slots.numpy()):
            if s >= 0:
                cache.codes[s // P, :, :, s % P], cache.words[s // P, :, :, s % P] = RL.packed(c[m]), w[m]
        out.copy_(torch.from_numpy(np.ascontiguousarray(t[:, :HEADS])))
        return out

    @staticmethod
    def aq_attn_kv4(q, cache, table, kv_len, cu_q=None):
        o = RL.attention(q.numpy(), cache.codes, cache.words, table.numpy(), kv_len.numpy(), None if cu_q is None else cu_q.numpy())
        return torch.from_numpy(o.astype(np.float32))


@pytest.fixture
def oracle(monkeypatch):
    for name in [n for n in vars(Oracle) if n.startswith("aq_")]:
        monkeypatch.setattr(mdl, name, getattr(Oracle, name))


def weights(seed, rope):
    rng = np.random.default_rng(seed)
    w = [{n: rng.standard_normal(s) * 0.02 for n, s in GEOMETRY.items()} for _ in range(LAYERS)]
    norms = [(rng.random(H) + 0.5).astype(np.float32) for _ in range(2 * LAYERS + 1)]
    r = SimpleNamespace(freq=(1e4 ** -(np.arange(D // 2) / (D // 2))).astype(np.float32), parts=(D // 2,)) if rope else None
    return w, norms, r


def decoder_of(w, norms, r):
    model = SimpleNamespace(layers=[{n: packed(W) for n, W in layer.items()} for layer in w])
    t = [torch.from_numpy(n) for n in norms]
    return mdl.Decoder(model, t[0:2 * LAYERS:2], t[1:2 * LAYERS:2], t[-1], r, HEADS, KV, D, EPS)


def batch(n_old, n_new):
    """(positions, slots, table, kv_len, cu_q) of sequences with n_old cached tokens and n_new new ones."""
    rng = np.random.default_rng(1)
    B = len(n_old)
    width = -(-int((n_old + n_new).max()) // P)
    table = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    pos = np.concatenate([a + np.arange(k) for a, k in zip(n_old, n_new)]).astype(np.int32)
    seq = np.repeat(np.arange(B), n_new)
    slots = table[seq, pos // P].astype(np.int64) * P + pos % P
    return [torch.from_numpy(np.ascontiguousarray(a)) for a in
            (pos, slots, table, (n_old + n_new).astype(np.int32), np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32))]


@pytest.mark.parametrize("caches", [0, LAYERS - 1, LAYERS + 1])
def test_a_cache_for_each_layer(oracle, caches):
    """Another number of caches than of layers is refused: layers are not left out."""
    dec = decoder_of(*weights(0, False))
    pos, slots, table, lens, cu = batch(np.array([0]), np.array([5]))
    with pytest.raises(ValueError, match="cache"):
        dec.step(torch.randn(5, H), [cache_of(table.numel()) for _ in range(caches)], pos, slots, table, lens, cu)
