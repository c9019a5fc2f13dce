"""What is not finite stays visible through a whole decoder (model.Decoder): a cached key
or value of NaN ends as NaN in the rows of its own sequence, and in no others' bits."""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
from tests.parity import to_dev
from tests.test_gpu_decoder import H, KV, LAYERS, P, decoder
from tests.test_gpu_layer import acts, dev, host, same_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(1, 64), (3, 4096), (5, 32768), (3, 32832), (256, 4096), (300, 20480), (257, 20544)])
def test_marked_rows(M, K):
    rng = np.random.default_rng(M + K)
    X = acts(rng, M, K)
    want = aq.aq_quant_act(dev(X))
    q, s = aq.aq_quant_act(dev(X), mark=True)
    same_rows(q, s, X)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
    bad = {0: np.nan, M // 2: np.inf, M - 1: -np.nan}
    for m, x in bad.items():
        X[m, (7 * m + K - 1) % K] = x
    keep = [m for m in range(M) if m not in bad]
    q, s = aq.aq_quant_act(dev(X), mark=True)
    assert not np.isfinite(host(s)[list(bad)]).any()
    assert torch.equal(q[keep], want[0][keep]) and torch.equal(s[keep], want[1][keep])


@pytest.mark.parametrize("kv", [0, 1], ids=["key", "value"])
@pytest.mark.parametrize("new", [None, [2, 80, 3], [1, 3, 2]], ids=["tokens", "chunks", "few"])
def test_a_cached_vector_that_is_not_finite(kv, new):
    dec, rng = decoder(11), np.random.default_rng(12)
    old, width = np.array([70, 41, 23]), 10
    pages = 3 * width + 2
    t = rng.permutation(pages)[:3 * width].astype(np.int32).reshape(3, width)
    clean = dec.caches(pages, P)

    def run(caches, at, n, cu):
        pos = np.concatenate([a + np.arange(k) for a, k in zip(at, n)])
        seq = np.repeat(np.arange(3), n)
        x = torch.randn((len(pos), H), generator=torch.Generator(device="cuda").manual_seed(len(pos)), device="cuda")
        slots = t[seq, pos // P].astype(np.int64) * P + pos % P
        return seq, dec.step(x, caches, to_dev(pos.astype(np.int32)), to_dev(slots), to_dev(t), to_dev((at + n).astype(np.int32)),
                             to_dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)) if cu else None)

    run(clean, 0 * old, old, True)
    n = np.ones(3, int) if new is None else np.array(new)
    for layer in range(LAYERS):
        caches = [aq.aq_kv4_cache_of(c.codes.clone(), c.words.clone()) for c in clean]
        token, head = 17, layer % KV
        caches[layer].words[t[1, token // P], kv, head, token % P] = 0x7FC00000
        again = [aq.aq_kv4_cache_of(c.codes.clone(), c.words.clone()) for c in clean]
        seq, (qx, sx, h) = run(again, old, n, new is not None)
        _, (bad_qx, bad_sx, bad_h) = run(caches, old, n, new is not None)
        assert np.isfinite(host(sx)).all() and np.isfinite(host(h)).all()
        hit = torch.from_numpy(seq == 1).cuda()
        assert not torch.isfinite(bad_sx[hit]).any() and torch.isnan(bad_h[hit]).all()
        assert torch.equal(bad_sx[~hit], sx[~hit]) and torch.equal(bad_qx[~hit], qx[~hit]) and torch.equal(bad_h[~hit], h[~hit])
        # what the other sequences appended is the same too
        for a, b in zip(caches, again):
            for b_ in (0, 2):
                at = t[b_].astype(np.int64)
                assert torch.equal(a.words[at], b.words[at]) and torch.equal(a.codes[at], b.codes[at])


def test_the_plain_quantizer_loses_the_mark():
    """The plain quantizer of the same rows gives 1e-12 for NaN, which is why the layer takes the marked one."""
    X = np.ones((2, 64), np.float32)
    X[1, 5] = np.nan
    assert host(aq.aq_quant_act(dev(X))[1])[1] == np.float32(1e-12)
    assert np.isnan(host(aq.aq_quant_act(dev(X), mark=True)[1])[1])
