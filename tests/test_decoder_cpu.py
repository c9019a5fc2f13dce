"""model.Decoder without a GPU: its calls answered by the FP64 oracle, so that what it joins to what shows."""
from types import SimpleNamespace
from unittest.mock import MagicMock

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
    def aq_workspace_bytes(pw, M, phase):
        return 0

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


# ---------------------------------------------------------------- what is joined to what

def product(q, s, W):
    return (s.astype(np.float32)[:, None] * (q.astype(np.int8).astype(np.float64) @ W.T)).astype(np.float32)


def reference(x, w, norms, r, cache, pos, slots, table, lens, cu, wrong=""):
    """A decoder written out: pre-norm layers whose residual sum is taken in FP32 behind each
    projection.  `wrong` plants a mistake."""
    f = np.float32
    x = x.astype(f)
    for l in range(LAYERS):
        na, nf = norms[2 * l], norms[2 * l + 1]
        if wrong == "norms swapped":
            na, nf = nf, na
        if wrong == "layer's weights" and l == 2:
            w = [w[0], w[1], w[1]]
        qkv = product(*RL.quant(RL.norm(x, na, None, EPS)[1]), w[l]["qkv"]).reshape(len(x), -1, D)
        turned = qkv[:, :HEADS + KV] if r is None else RL.rope(qkv[:, :HEADS + KV], pos[None], r.freq, r.parts)
        c, ws = RL.hold(np.stack([turned[:, HEADS:], qkv[:, HEADS + KV:]], 1))
        for m, s in enumerate(slots):
            cache[l].codes[s // P, :, :, s % P], cache[l].words[s // P, :, :, s % P] = RL.packed(c[m]), ws[m]
        a = RL.attention(turned[:, :HEADS], cache[l].codes, cache[l].words, table, lens, cu).astype(f)
        o = product(*RL.quant(a), w[l]["o"])
        mid = o if wrong == "no residual" and l == 1 else o + x
        y = RL.norm(x if wrong == "stale rows" else mid, nf, None, EPS)[1]
        gate = RL.swiglu(product(*RL.quant(y), w[l]["gate_up"]))
        x = product(*RL.quant(gate), w[l]["down"]) + (x if wrong == "residual in front of attention" else mid)
    return (*RL.quant(RL.norm(x, norms[-1], None, EPS)[1]), x)


def both(rope, wrong="", seed=3):
    w, norms, r = weights(seed, rope)
    dec = decoder_of(w, norms, r)
    rng = np.random.default_rng(seed + 1)
    same = True
    old = np.array([0, 0, 0])
    new = [np.array([70, 1, 9]), np.array([1, 1, 1]), np.array([2, 5, 1])]      # a prompt, tokens, chunks
    pages = 3 * 8
    mine, theirs = ([cache_of(pages) for _ in range(LAYERS)] for _ in range(2))
    table = rng.permutation(pages).astype(np.int32).reshape(3, 8)
    for n in new:
        pos = np.concatenate([a + np.arange(k) for a, k in zip(old, n)]).astype(np.int32)
        seq = np.repeat(np.arange(3), n)
        slots = table[seq, pos // P].astype(np.int64) * P + pos % P
        old = old + n
        cu = None if (n == 1).all() else np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        x = rng.standard_normal((len(pos), H)).astype(np.float32)
        t = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)) for a in (x, pos, slots, table, old.astype(np.int32), cu)]
        kept = t[0].clone()
        q, s, h = dec.step(t[0], mine, *t[1:])
        assert torch.equal(t[0], kept)                       # the caller's rows
        rq, rs, rh = reference(x, w, norms, r, theirs, pos, slots, table, old, cu, wrong)
        same &= np.array_equal(h.numpy(), rh) and np.array_equal(q.numpy(), rq) and np.array_equal(s.numpy(), rs.astype(np.float32))
        same &= all(np.array_equal(a.codes, b.codes) and np.array_equal(a.words, b.words) for a, b in zip(mine, theirs))
    return same


@pytest.mark.parametrize("rope", [True, False], ids=["rope", "none"])
def test_layers_written_out(oracle, rope):
    """Prompts, single tokens and chunks on one cache: the rows, codes and caches of a decoder that is
    written out, to the bit."""
    assert both(rope)


@pytest.mark.parametrize("wrong", ["norms swapped", "layer's weights", "no residual", "stale rows", "residual in front of attention"])
def test_planted_mistakes_are_seen(oracle, wrong):
    assert not both(True, wrong)


# ---------------------------------------------------------------- workspaces

def test_a_workspace_for_each_step(oracle, monkeypatch):
    """The decode kernels' workspace is the step's own, large enough for each of its projections, its counters zero
    at first: the stream's would be shared by graphs captured on one stream, and be freed under them where a call of
    more rows needs a larger one."""
    need = lambda pw, M, phase: 0 if M < 4 else (1 << 18) + 64 * M + pw.K   # noqa: E731
    seen = []

    def decode(pw, qx, sx, out=None, ws=None):
        M = qx.shape[0]
        if need(pw, M, 0):
            assert ws is not None and ws.dtype == torch.uint8 and ws.numel() >= need(pw, M, 0)
            assert (ws[:1 << 18] == 0).all()                 # (as every call leaves them)
        seen.append(ws)
        return Oracle.aq_linear_decode(pw, qx, sx, out)

    monkeypatch.setattr(mdl, "aq_workspace_bytes", need)
    monkeypatch.setattr(mdl, "aq_linear_decode", decode)
    dec = decoder_of(*weights(0, False))
    steps = []
    for n in (5, 5, 9, 5, 3, 64, 65):
        seen.clear()
        pos, slots, table, lens, cu = batch(np.array([0]), np.array([n]))
        dec.step(torch.randn(n, H), [cache_of(table.numel()) for _ in range(LAYERS)], pos, slots, table, lens, cu)
        assert len(seen) == (4 * LAYERS if n <= 64 else 0) and len({id(w) for w in seen}) <= 1
        if 4 <= n <= 64:
            steps.append(seen[0])
    assert len({w.data_ptr() for w in steps}) == len(steps)   # (all held here: none is another's)
    pos, slots, table, lens, cu = batch(np.array([0]), np.array([5]))
    seen.clear()
    dec.layer(0, torch.randn(5, H), None, cache_of(table.numel()), pos, slots, table, lens, cu)
    assert len(seen) == 4 and seen[0] is not None and len({id(w) for w in seen}) == 1


# ---------------------------------------------------------------- devices

@pytest.mark.parametrize("here", [0, 1])
@pytest.mark.parametrize("M", [3, 65])
def test_on_the_device_of_the_rows(monkeypatch, here, M):
    """Every call of a layer and of linear runs with the rows' device current, whichever was."""
    current, made = [here], []

    class Made:
        def __init__(self, device):
            self.device, self.before = device, None

        def __enter__(self):
            self.before, current[0] = current[0], self.device.index

        def __exit__(self, *e):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Made)
    rows = MagicMock(shape=(M, H), device=torch.device("cuda", 1))
    rows.unflatten.return_value.__getitem__.return_value = rows

    def call(n):
        def f(*a, **k):
            made.append(current[0])
            return (rows,) * n if n > 1 else rows
        return f

    for name, n in (("aq_norm_quant", 3), ("aq_quant_act", 2), ("aq_rope_kv4", 1), ("aq_attn_kv4", 1), ("aq_swiglu_quant", 2),
                    ("aq_linear_decode", 1), ("aq_linear_prefill", 1)):
        monkeypatch.setattr(mdl, name, call(n))
    monkeypatch.setattr(mdl, "aq_workspace_bytes", lambda *a: 0)
    dec = decoder_of(*weights(0, False))
    dec.layer(0, rows, rows, None, None, None, None, None)
    mdl.linear(None, rows, rows)
    assert made == [1] * 11 and current == [here]
