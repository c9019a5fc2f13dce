"""The per-token-factor operators where the order of a sum, a position or a
value that is not finite could show: beside test_gpu_routed.py, whose helpers
and tolerances these use."""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
from tests.parity import say, to_dev
from tests.test_gpu_routed import bf16, host
from workloads import gen

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- router: equal experts, permuted tokens

def check_equal_experts(ids, w, group, name):
    """Of experts with equal rows the lower ones come first, next to each
    other, with equal weights bit for bit; no tolerance."""
    for m in range(len(ids)):
        g = group[ids[m]]
        for v in np.unique(g):
            at = np.flatnonzero(g == v)
            assert (np.diff(at) == 1).all(), f"{name}: token {m} {ids[m].tolist()}"
            assert np.array_equal(ids[m, at], np.flatnonzero(group == v)[: len(at)]), f"{name}: token {m} {ids[m].tolist()}"
            assert len(np.unique(w[m, at].view(np.int32))) == 1, f"{name}: token {m} {w[m, at].tolist()}"


# real values, whose FP64 sums are rounded, so that another order of sums shows
@pytest.mark.parametrize("M,K,E,dist,wtype,score", [
    (40, 2048, 64, 16, "f32", "softmax"),
    (64, 2048, 64, 32, "bf16", "sigmoid"),
    (64, 704, 70, 1, "f32", "softmax"),
    (37, 4096, 250, 16, "f32", "sigmoid"),
    (160, 1024, 128, 48, "bf16", "softmax"),
    (1024, 1024, 160, 16, "bf16", "softmax"),
    (700, 320, 1000, 17, "f32", "softmax"),
    (9, 2048, 64, 16, "f32", "softmax"),       # a wave per token and expert
])
def test_route_equal_experts(M, K, E, dist, wtype, score):
    """Expert e + dist repeats expert e: equal keys, whatever place of a tile
    either has."""
    rng = np.random.default_rng(M + E)
    X = gen.acts_outliers(rng, M, K, max(1, K // 100), 30.0)
    group = np.arange(E)
    group = np.where(group // dist % 2 == 1, group - dist, group)
    W = (rng.standard_normal((E, K)) * 0.4 / np.sqrt(K)).astype(np.float32)[group]
    Wd = bf16(W).cuda() if wtype == "bf16" else to_dev(W)
    ids, w = aq.aq_moe_route(to_dev(X), Wd, 8, score=score)
    say(f"  M{M} E{E} distance {dist}")
    check_equal_experts(host(ids), host(w), group, f"M{M} E{E} distance {dist}")


@pytest.mark.parametrize("M,K,E", [(48, 2048, 64), (37, 4096, 250), (333, 704, 96), (1024, 1024, 160), (12, 512, 100)])
def test_route_permuted_tokens(M, K, E):
    """A token's experts and weights do not depend on its row: tokens in another
    order, and the same token in several rows (the experts in equal pairs, so
    that one last bit of a sum shows)."""
    rng = np.random.default_rng(M)
    X = gen.acts_outliers(rng, M, K, max(1, K // 100), 30.0)
    h = M // 2
    X[M - h:] = X[:h]
    group = np.arange(E) // 32 * 32 + np.arange(E) % 16
    W = to_dev((rng.standard_normal((E, K)) * 0.4 / np.sqrt(K)).astype(np.float32)[group])
    ids, w = (host(t) for t in aq.aq_moe_route(to_dev(X), W, 6))
    check_equal_experts(ids, w, group, f"M{M} E{E}")
    assert np.array_equal(ids[M - h:], ids[:h]) and np.array_equal(w[M - h:].view(np.int32), w[:h].view(np.int32))
    for perm in (np.roll(np.arange(M), 16), np.roll(np.arange(M), 1), rng.permutation(M)):
        i2, w2 = (host(t) for t in aq.aq_moe_route(to_dev(X[perm]), W, 6))
        assert np.array_equal(i2, ids[perm])
        assert np.array_equal(w2.view(np.int32), w[perm].view(np.int32))
