"""A whole decoder over packed projections (model.Decoder): every step between
the projections against its definition on the rows that the layer itself gave it, a
prompt and then single tokens, and its captured form."""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
import mixed_precision_int_amd.model as mdl
from oracle import layer as RL
from tests.test_gpu_layer import check_attn, freqs, host, same_rows
from tests.parity import to_dev

pytestmark = pytest.mark.gpu

H, I, HEADS, KV, D, LAYERS, P = 256, 384, 4, 2, 64, 2, 16
GEOMETRY = [("qkv", (HEADS + 2 * KV) * D, H), ("o", H, HEADS * D), ("gate_up", 2 * I, H), ("down", H, I)]


def decoder(seed=0, rope=True):
    rng = np.random.default_rng(seed)
    maps = [[rng.choice([4, 8], size=(N // 64, K // 128)) for _, N, K in GEOMETRY] for _ in range(LAYERS)]
    model = mdl.pack_model(GEOMETRY, maps, lambda l, name, N, K: to_dev((rng.standard_normal((N, K)) * 0.05).astype(np.float32)))
    norm = lambda: to_dev((rng.random(H) + 0.5).astype(np.float32))  # noqa: E731
    r = aq.aq_rope_axes(to_dev(freqs(D // 2, 1e4)), (D // 2,), D) if rope else None
    return mdl.Decoder(model, [norm() for _ in range(LAYERS)], [norm() for _ in range(LAYERS)], norm(), r, HEADS, KV, D)


class Watch:
    """The calls that a layer makes, with what went in and out."""

    def __init__(self, monkeypatch):
        self.seen = []
        for name in ("aq_norm_quant", "aq_rope_kv4", "aq_attn_kv4", "aq_swiglu_quant", "aq_quant_act"):
            monkeypatch.setattr(mdl, name, self.wrap(name, getattr(aq, name)))

    def wrap(self, name, f):
        def call(*a, **k):
            a = [t.clone() if isinstance(t, torch.Tensor) else t for t in a]
            before = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in k.items()}
            if name == "aq_rope_kv4":
                before["rows"] = a[0].clone()
                k["out"] = a[0].unflatten(1, (-1, D))[:, :HEADS]
            if k.get("h") is not None:
                k["h"] = k["residual"] = k["h"].clone()
            r = f(*a, **k)
            torch.cuda.synchronize()
            self.seen.append((name, a, before, [t.clone() for t in (r if isinstance(r, tuple) else (r,))]))
            return r
        return call


def test_every_step_of_a_prompt_and_of_tokens(monkeypatch):
    dec, rng = decoder(), np.random.default_rng(5)
    new = [70, 1, 23]
    width = 8
    table = torch.randperm(3 * width + 2, device="cuda")[:3 * width].int().view(3, width)
    caches = dec.caches(3 * width + 2, P)
    assert len(caches) == LAYERS and caches[0].heads == KV and caches[0].D == D
    lens = np.array(new)
    for turn in range(3):
        if turn == 0:
            pos = np.concatenate([np.arange(n) for n in new])
            seq = np.repeat(np.arange(3), new)
            cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        else:
            pos, seq, cu = lens.copy(), np.arange(3), None
            lens = lens + 1
        t = host(table)
        slots = t[seq, pos // P].astype(np.int64) * P + pos % P
        x = torch.randn((len(pos), H), device="cuda") * 2
        kept = x.clone()
        with monkeypatch.context() as m:
            w = Watch(m)
            qx, sx, h = dec.step(x, caches, to_dev(pos.astype(np.int32)), to_dev(slots), table, to_dev(lens.astype(np.int32)),
                                 None if cu is None else to_dev(cu))
        assert torch.equal(x, kept)
        assert qx.dtype == torch.int8 and qx.shape == (len(pos), H) and h.shape == qx.shape and torch.isfinite(h).all()
        names = [s[0] for s in w.seen]
        assert names == ["aq_norm_quant", "aq_rope_kv4", "aq_attn_kv4", "aq_quant_act", "aq_norm_quant", "aq_swiglu_quant"] * LAYERS + \
            ["aq_norm_quant"]
        layer = 0
        for name, a, k, r in w.seen:
            if name == "aq_norm_quant":
                res = k.get("residual")
                hh, y = RL.norm(host(a[0]), host(a[1]), None if res is None else host(res), dec.eps)
                same_rows(r[0], r[1], y, name)
                if res is not None:
                    assert np.array_equal(host(r[2]), hh)
            elif name == "aq_swiglu_quant":
                same_rows(r[0], r[1], RL.swiglu(host(a[0])))
            elif name == "aq_quant_act":
                same_rows(r[0], r[1], host(a[0]))
                layer += 1
            elif name == "aq_rope_kv4":
                rows = host(k["rows"]).reshape(len(pos), -1, D)
                q = RL.rope(rows[:, :HEADS + KV], [pos], host(dec.rope.freq), dec.rope.parts)
                assert np.array_equal(host(r[0]), q[:, :HEADS])
                c, ws = RL.hold(np.stack([q[:, HEADS:], rows[:, HEADS + KV:]], 1))
                cache = caches[layer]
                assert np.array_equal(host(cache.words).view(np.uint32)[slots // P, :, :, slots % P], ws)
                assert np.array_equal(host(cache.codes)[slots // P, :, :, slots % P], RL.packed(c))
            else:
                codes, words = host(caches[layer].codes), host(caches[layer].words).view(np.uint32)
                check_attn(host(a[0]), codes, words, t, lens, cu, name=f"turn {turn} layer {layer}", got=r[0])


def test_captured_and_shapes():
    dec = decoder(3)
    caches = dec.caches(8, P)
    table, lens = torch.arange(8, device="cuda").int().view(2, 4), to_dev(np.array([33, 9], np.int32))
    pos, slots = to_dev(np.array([32, 8], np.int32)), to_dev(np.array([2 * P, 4 * P + 8], np.int64))
    x = torch.randn((2, H), device="cuda")
    eager = [t.clone() for t in dec.step(x, caches, pos, slots, table, lens)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        dec.step(x, caches, pos, slots, table, lens)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        outs = dec.step(x, caches, pos, slots, table, lens)
    for _ in range(3):
        for t in outs:
            t.zero_()
        g.replay()
        again = dec.step(x, caches, pos, slots, table, lens)
        torch.cuda.synchronize()
        for a, b, c in zip(outs, again, eager):
            assert torch.equal(a, c) and torch.equal(b, c)
    with pytest.raises(ValueError):
        mdl.Decoder(dec.model, dec.attn_norms, dec.ffn_norms, dec.final_norm, dec.rope, HEADS, KV + 1, D)
    with pytest.raises(ValueError):
        mdl.Decoder(dec.model, dec.attn_norms[:1], dec.ffn_norms, dec.final_norm, dec.rope, HEADS, KV, D)
