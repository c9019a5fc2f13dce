"""A decoder's calls on the GPU in their order: each takes the weights of its layer and what the call
before it gave, and each packed projection is the oracle's on either side of the rows where the
decode kernels give way to the prefill ones."""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
import mixed_precision_int_amd.model as mdl
from oracle import aq_oracle as O
from tests.parity import assert_output_close, to_dev
from tests.test_gpu_decoder import D, GEOMETRY, H, HEADS, KV, LAYERS, P
from tests.test_gpu_layer import check_attn, freqs, host

pytestmark = pytest.mark.gpu

CALLS = ("aq_norm_quant", "aq_rope_kv4", "aq_attn_kv4", "aq_swiglu_quant", "aq_quant_act", "aq_linear_decode", "aq_linear_prefill")


def watch(monkeypatch, seen):
    def wrap(name, f):
        def call(*a, **k):
            held = {i: t.clone() for i, t in [*enumerate(a), *k.items()] if isinstance(t, torch.Tensor)}
            r = f(*a, **k)
            torch.cuda.synchronize()
            seen.append((name, a, k, held, [t.clone() for t in (r if isinstance(r, tuple) else (r,))]))
            return r
        return call
    for name in CALLS:
        monkeypatch.setattr(mdl, name, wrap(name, getattr(aq, name)))


@pytest.mark.parametrize("rope", [True, False], ids=["rope", "none"])
@pytest.mark.parametrize("new", [None, [60, 1, 3], [61, 3, 1], [200, 9, 70]], ids=["3", "64", "65", "279"])
def test_calls_in_their_order(monkeypatch, new, rope):
    rng = np.random.default_rng(31)
    maps = [[rng.choice([4, 8], size=(N // 64, K // 128)) for _, N, K in GEOMETRY] for _ in range(LAYERS)]
    W = [[(rng.standard_normal((N, K)) * 0.05).astype(np.float32) for _, N, K in GEOMETRY] for _ in range(LAYERS)]
    at = {name: i for i, (name, _, _) in enumerate(GEOMETRY)}
    model = mdl.pack_model(GEOMETRY, maps, lambda l, name, N, K: to_dev(W[l][at[name]]))
    norms = [to_dev((rng.random(H) + 0.5).astype(np.float32)) for _ in range(2 * LAYERS + 1)]
    r = aq.aq_rope_axes(to_dev(freqs(D // 2, 1e4)), (D // 2,), D) if rope else None
    dec = mdl.Decoder(model, norms[0:-1:2], norms[1:-1:2], norms[-1], r, HEADS, KV, D)
    old, n = np.array([40, 3, 17]), np.ones(3, int) if new is None else np.array(new)
    width = -(-int((old + n).max()) // P)
    table = rng.permutation(3 * width).astype(np.int32).reshape(3, width)
    caches = dec.caches(3 * width, P)
    for c in caches:                                    # cached tokens: anything that is finite
        c.codes.random_(0, 256)
        c.words.copy_((torch.rand(c.words.shape, device="cuda") + 0.5).view(torch.int32) & ~15 | 7)
    pos = np.concatenate([a + np.arange(k) for a, k in zip(old, n)]).astype(np.int32)
    seq = np.repeat(np.arange(3), n)
    slots = table[seq, pos // P].astype(np.int64) * P + pos % P
    x = torch.randn((len(pos), H), device="cuda") * 2
    seen = []
    watch(monkeypatch, seen)
    given = [to_dev(a) for a in (pos, slots, table, (old + n).astype(np.int32))]
    cu = None if new is None else np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q, s, h = dec.step(x, caches, *given, None if cu is None else to_dev(cu))
    calls = iter(seen)
    linear = "aq_linear_decode" if len(pos) <= mdl.DECODE_ROWS else "aq_linear_prefill"

    def norm(w, X, residual):
        name, a, k, held, out = next(calls)
        assert name == "aq_norm_quant" and a[1] is w and k.get("eps") == dec.eps and torch.equal(held[0], X)
        assert (k.get("residual") is None) == (residual is None) and (residual is None or torch.equal(held["residual"], residual))
        return out[0], out[1], X if residual is None else out[2]

    def project(l, which, qx, sx):
        name, a, k, held, out = next(calls)
        assert name == linear and a[0] is model.layers[l][which] and torch.equal(held[1], qx) and torch.equal(held[2], sx)
        codes, sW = O.quant_weights(W[l][at[which]], maps[l][at[which]], 64, 128)
        part = O.tile_partials(host(qx).astype(np.int64), codes, 128)
        sx = host(sx).astype(np.float64)
        assert_output_close(host(out[0]), O.linear_from_partials(part, sx, sW), O.abs_contrib(part, sx, sW), f"{l} {which}")
        return out[0]

    rows, delta = x, None
    for l in range(LAYERS):
        qx, sx, rows = norm(norms[2 * l], x, None) if delta is None else norm(norms[2 * l], delta, rows)
        qkv = project(l, "qkv", qx, sx)
        name, a, k, held, out = next(calls)
        assert name == "aq_rope_kv4" and torch.equal(held[0], qkv) and a[1] is r and a[2] is given[0] and a[3] is caches[l] and a[4] is given[1]
        name, a, k, held, att = next(calls)
        assert name == "aq_attn_kv4" and torch.equal(held[0], out[0]) and a[1] is caches[l] and a[2] is given[2] and a[3] is given[3]
        check_attn(host(held[0]), host(caches[l].codes), host(caches[l].words).view(np.uint32), table, old + n, cu, name=f"layer {l}", got=att[0])
        name, a, k, held, out = next(calls)
        assert name == "aq_quant_act" and torch.equal(held[0], att[0]) and k == {"mark": True}
        o = project(l, "o", *out)
        qx, sx, rows = norm(norms[2 * l + 1], o, rows)
        y = project(l, "gate_up", qx, sx)
        name, a, k, held, out = next(calls)
        assert name == "aq_swiglu_quant" and torch.equal(held[0], y)
        delta = project(l, "down", *out)
    out = norm(norms[-1], delta, rows)
    assert next(calls, None) is None
    assert torch.equal(q, out[0]) and torch.equal(s, out[1]) and torch.equal(h, out[2])
