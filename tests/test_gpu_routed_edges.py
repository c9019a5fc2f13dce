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


# ---------------------------------------------------------------- router: logits that are not finite

@pytest.mark.parametrize("M,E,k", [(6, 16, 3), (8, 100, 5), (6, 300, 4), (80, 64, 6), (40, 1000, 8), (1100, 40, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_not_finite(M, E, k, score, norm):
    """A token of NaN or infinities has ids in range, without excluded experts,
    and weights that show it; the other tokens are as they were."""
    rng = np.random.default_rng(E)
    K = 128
    X = gen.acts_outliers(rng, M, K, 2, 30.0)
    W = (rng.standard_normal((E, K)) * 0.05).astype(np.float32)
    W[:, 5] = np.where(rng.random(E) < 0.5, 1, -1) * (np.abs(W[:, 5]) + 0.01)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    out = rng.permutation(E)[: E // 4]
    bias[out] = -np.inf
    W[np.setdiff1d(np.arange(E), out)[: k + 1], 5] = 0.01      # k + 1 experts with a logit of +inf at least
    clean_ids, clean_w = (host(t) for t in aq.aq_moe_route(to_dev(X), to_dev(W), k, to_dev(bias), score, norm))
    X[1, 7], X[2, 5], X[3, 7] = np.nan, np.inf, -np.float32(np.nan)
    X[3, 9], X[M - 1, :] = np.inf, np.nan
    bad = np.array([1, 2, 3, M - 1])
    ids, w = (host(t) for t in aq.aq_moe_route(to_dev(X), to_dev(W), k, to_dev(bias), score, norm))
    good = np.setdiff1d(np.arange(M), bad)
    assert np.array_equal(ids[good], clean_ids[good])
    assert np.array_equal(w[good].view(np.int32), clean_w[good].view(np.int32))
    # every key of tokens 1, 3 and M - 1 is NaN: the lowest experts that are not excluded
    left = np.setdiff1d(np.arange(E), out)
    for m in (1, 3, M - 1):
        assert np.array_equal(ids[m], left[:k]) and np.isnan(w[m]).all(), (m, ids[m], w[m])
    # token 2: logits of +inf and -inf
    plus = left[W[left, 5] > 0]
    assert np.isin(ids[2], plus).all() and len(np.unique(ids[2])) == k
    if score == "softmax":
        assert np.isnan(w[2]).all()
    else:                                        # p = 1 each
        assert np.abs(w[2] - (1 / k if norm else 1)).max() <= 2.0 ** -24


@pytest.mark.parametrize("M", [1, 2, 5, 9, 200])
def test_layer_not_finite(M):
    """The layer's outputs of a NaN token are NaN, not zeros; the others' stay."""
    from tests.test_gpu_routed import Experts
    rng = np.random.default_rng(M)
    ex = Experts(12, 512, 128, seed=2)
    X = gen.acts_outliers(rng, M, 512, 5, 30.0)
    Wr = to_dev((rng.standard_normal((12, 512)) * 0.05).astype(np.float32))
    want, _, _ = aq.aq_moe_layer(ex.dev, to_dev(X), Wr, 3)
    X[M // 2, 100] = np.nan
    Y, ids, w = aq.aq_moe_layer(ex.dev, to_dev(X), Wr, 3)
    Y, want = host(Y), host(want)
    assert np.isnan(Y[M // 2]).all() and np.isnan(host(w)[M // 2]).all()
    assert ((host(ids) >= 0) & (host(ids) < 12)).all()
    keep = np.arange(M) != M // 2
    assert np.array_equal(Y[keep], want[keep])


# ---------------------------------------------------------------- adapters: values that are not finite

def by_rows(M, L, K, N, R, t):
    """Whether a call takes the tokens one by one (else in tiles of one adapter)."""
    n = M * R * (K + N) * (4 if t == "f32" else 2)
    return n < 128 << 20 or (M <= L and n <= 192 << 20)


def tokens_for_tiles(K, N, R, t):
    return (128 << 20) // (R * (K + N) * (4 if t == "f32" else 2)) + 5


def check_adapters(got, Y, X, ids, A, B, sc, ranks, rows):
    """The named rows against the definition in 64 bits: infinities and NaN the
    same, the rest within the FP32 products and sums over K, at most 16 column
    ranges, R, the scale and the last addition: (K + R + 20) u of the sum of the
    terms' magnitudes."""
    A, B = A.astype(np.float64), B.astype(np.float64)
    for m in rows:
        y, mag = Y[m].astype(np.float64), np.abs(Y[m].astype(np.float64))
        a = ids[m]
        with np.errstate(invalid="ignore"):
            if 0 <= a < len(A):
                r = min(max(int(ranks[a]), 0), A.shape[1])
                x = X[m].astype(np.float64)
                v = (A[a, :r] * x).sum(1)
                y = y + float(sc[a]) * (B[a, :, :r] * v).sum(1)
                mag = mag + abs(float(sc[a])) * (np.abs(B[a, :, :r]) * np.abs(A[a, :r] * x).sum(1)).sum(1)
            g = got[m].astype(np.float64)
            assert np.array_equal(np.isnan(g), np.isnan(y)), f"token {m}, adapter {a}: {g[:6]} {y[:6]}"
            assert np.array_equal(g[np.isinf(y)], y[np.isinf(y)]), f"token {m}, adapter {a}: {g[:6]} {y[:6]}"
            f = np.isfinite(y)
            assert (np.abs(g[f] - y[f]) <= (X.shape[1] + A.shape[1] + 20) * 2.0 ** -24 * mag[f] + 1e-30).all(), (m, a)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,K,N", [(8, 1024, 2048), (16, 512, 1024), (24, 1088, 960), (64, 704, 576), (128, 512, 576)])
@pytest.mark.parametrize("tiles", [False, True])
def test_lora_infinities(R, K, N, t, tiles):
    """Infinities in activations and adapters end where the definition puts them,
    whichever way a call's tokens are taken."""
    from tests.test_gpu_routed import TYPES
    L, M = 5, tokens_for_tiles(K, N, R, t) if tiles else 14
    assert by_rows(M, L, K, N, R, t) != tiles
    rng = np.random.default_rng(R)
    A = (rng.standard_normal((L, R, K)) / np.sqrt(K)).astype(np.float32)
    B = (rng.standard_normal((L, N, R)) * 0.1).astype(np.float32)
    sc = (rng.random(L) + 0.5).astype(np.float32)
    ranks = np.array([1, R, R, R - 2, 3], np.int32)
    A[0], B[0] = 0.5, np.abs(B[0]) + 0.01            # (0.5: one piece)
    A[1], B[1] = np.abs(A[1]) + 0.01, np.abs(B[1]) + 0.01
    A[2, 0, 7] = np.inf
    B[3, 30, 0] = np.inf
    B[3, 9, R - 3] = -np.inf
    A[4, :, 11] = 0                                  # 0 times infinity
    for a, r in enumerate(ranks):
        A[a, r:], B[a, :, r:] = np.nan, np.inf
    At, Bt = (torch.from_numpy(x).to(TYPES[t]) for x in (A, B))
    A, B = At.float().numpy(), Bt.float().numpy()
    X = gen.acts_outliers(rng, M, K, 5, 30.0)
    Y = rng.standard_normal((M, N)).astype(np.float32)
    ids = rng.integers(-1, L, M).astype(np.int32)
    at = rng.permutation(M)[:14]
    ids[at] = (0, 0, 0, 1, 1, 1, 2, 2, 3, 3, 4, 4, -1, 0)
    X[at[0], 5], X[at[1], K - 1], X[at[2], 6] = np.inf, -np.inf, np.nan
    X[at[3], 5], X[at[4], 70], X[at[5], [3, K - 9]] = np.inf, -np.inf, (np.inf, -np.inf)
    X[at[6], 7], X[at[7], 7] = 1.0, -2.0             # (one piece)
    X[at[8]] = np.where(np.abs(X[at[8]]) < 1, 1.0, -1.0)
    X[at[10], 11], X[at[11], 3], X[at[12], 0] = np.inf, np.inf, np.inf
    X[at[13]] = np.float32(1e38)                     # v is past FP32's range
    lora = aq.aq_lora_adapters(At.cuda(), Bt.cuda(), to_dev(sc), to_dev(ranks))
    say(f"  R{R} {t} M{M}")
    got = host(aq.aq_lora_add(lora, to_dev(X), to_dev(ids), to_dev(Y)))
    assert (got[at[13]] == np.inf).all()
    check_adapters(got, Y, X, ids, A, B, sc, ranks, np.setdiff1d(np.r_[at, rng.integers(0, M, 20)], at[13:]))


# ---------------------------------------------------------------- adapters: tokens in tiles
# (the sizes are such that the call groups its tokens: by_rows() is false)

def device_pool(seed, L, R, K, N, t):
    """A pool made on the device, ranks 0 .. R, NaN and infinities beyond them."""
    from tests.test_gpu_routed import TYPES
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = (torch.randn((L, R, K), generator=g, device="cuda") / K ** 0.5).to(TYPES[t])
    B = (torch.randn((L, N, R), generator=g, device="cuda") * 0.1).to(TYPES[t])
    sc = torch.rand(L, generator=g, device="cuda") + 0.5
    ranks = torch.randint(0, R + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
    ranks[0] = R
    beyond = torch.arange(R, device="cuda")[None, :] >= ranks[:, None]
    A[beyond] = float("nan")
    B.transpose(1, 2)[beyond] = float("inf")
    return A, B, sc, ranks


def check_rows(got, Y, X, ids, pool, rows):
    """check_adapters for some rows, with the adapters that they have."""
    A, B, sc, ranks = pool
    used = np.unique(ids[rows])
    used = used[(used >= 0) & (used < len(A))]
    sel = torch.from_numpy(used).long().cuda()
    a, b, s, r = (host(x[sel].float() if x.dtype != torch.int32 else x[sel]) for x in (A, B, sc, ranks))
    where = {u: i for i, u in enumerate(used)}
    here = np.array([where.get(int(i), -1) for i in ids])
    with np.errstate(invalid="ignore"):
        check_adapters(got, Y, X, here, a, b, s, r, rows)


@pytest.mark.parametrize("M,L,K,N,t", [
    (9000, 8192, 256, 768, "bf16"),      # more tokens than the grouping keeps in registers; 9 groups a thread
    (3000, 8192, 1024, 3264, "f16"),
    (4200, 1024, 256, 896, "f32"),       # one group more than threads
    (20000, 1500, 64, 512, "bf16"),
])
def test_lora_tiles_large_pools(M, L, K, N, t):
    """Pools up to the largest: a group of its own for every adapter, most of them
    of no token or one; some rows against the definition, all of them against the
    tokens in another order."""
    R = 8
    assert not by_rows(M, L, K, N, R, t)
    pool = device_pool(L, L, R, K, N, t)
    rng = np.random.default_rng(M)
    ids = rng.integers(-2, L + 2, M).astype(np.int32)
    ids[rng.random(M) < 0.2] = L - 1                   # and a full tile or more
    ids[:70] = 3
    X = gen.acts_outliers(rng, M, K, 2, 30.0)
    Y = rng.standard_normal((M, N)).astype(np.float32)
    lora = aq.aq_lora_adapters(*pool)
    say(f"  M{M} L{L} {t}")
    got = host(aq.aq_lora_add(lora, to_dev(X), to_dev(ids), to_dev(Y)))
    check_rows(got, Y, X, ids, pool, np.unique(np.r_[0, 69, M - 1, rng.integers(0, M, 60)]))
    none = (ids < 0) | (ids >= L)
    assert none.any() and np.array_equal(got[none], Y[none])
    perm = rng.permutation(M)
    again = host(aq.aq_lora_add(lora, to_dev(X[perm]), to_dev(ids[perm]), to_dev(Y[perm])))
    assert np.array_equal(again, got[perm])


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R", [8, 24, 64])
def test_lora_tiles_isolation(R, t):
    """A token of NaN or infinities, an adapter of them and what lies beyond a rank
    stay their own, in tiles that are full, nearly empty and of no adapter."""
    K, N, L = 832, 704, 5
    M = tokens_for_tiles(K, N, R, t)
    assert not by_rows(M, L, K, N, R, t)
    pool = device_pool(R, L, R, K, N, t)
    rng = np.random.default_rng(R)
    ids = rng.choice([-1, 0, 1, 2], M, p=[0.1, 0.5, 0.3, 0.1]).astype(np.int32)
    ids[[5, 77, M - 1]] = 3                            # a tile of three tokens
    X = gen.acts_outliers(rng, M, K, 5, 30.0)
    Y = rng.standard_normal((M, N)).astype(np.float32)
    lora = aq.aq_lora_adapters(*pool)
    say(f"  R{R} {t} M{M}")
    want = host(aq.aq_lora_add(lora, to_dev(X), to_dev(ids), to_dev(Y)))
    check_rows(want, Y, X, ids, pool, np.unique(np.r_[5, 77, M - 1, rng.integers(0, M, 40)]))
    bad = np.unique(np.r_[77, rng.integers(0, M, M // 5)])
    X2 = X.copy()
    X2[bad[::3]], X2[bad[1::3]], X2[bad[2::3], 11] = np.nan, -np.inf, np.inf
    other = np.setdiff1d(rng.integers(0, M, 30), [5, M - 1])
    ids2 = ids.copy()
    ids2[other] = 4
    pool[0][4], pool[1][4] = float("inf"), float("nan")
    got = host(aq.aq_lora_add(lora, to_dev(X2), to_dev(ids2), to_dev(Y)))
    keep = np.setdiff1d(np.arange(M), np.r_[bad, other])
    assert np.array_equal(got[keep], want[keep]) and len(keep) > M // 2


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R", [8, 40, 128])
def test_lora_tiles_slices_and_in_place(R, t):
    """Row strides other than N, of Yin and of Y, in place and apart; the columns
    and rows beside them stay as they were."""
    K, N, L = 704, 832, 4
    M = tokens_for_tiles(K, N, R, t)
    assert not by_rows(M, L, K, N, R, t)
    pool = device_pool(R + 1, L, R, K, N, t)
    lora = aq.aq_lora_adapters(*pool)
    rng = np.random.default_rng(R)
    ids = rng.integers(-1, L, M).astype(np.int32)
    X = gen.acts_outliers(rng, M, K, 5, 30.0)
    wide = rng.standard_normal((M + 2, N + 192)).astype(np.float32)
    Xd, idd, G = to_dev(X), to_dev(ids), to_dev(wide)
    part = G[1:-1, 64:64 + N]
    say(f"  R{R} {t} M{M}")
    ref = host(aq.aq_lora_add(lora, Xd, idd, part.contiguous()))
    check_rows(ref, wide[1:-1, 64:64 + N], X, ids, pool, np.unique(np.r_[0, M - 1, rng.integers(0, M, 30)]))
    assert np.array_equal(host(aq.aq_lora_add(lora, Xd, idd, part)), ref) and np.array_equal(host(G), wide)
    apart = torch.full((M + 2, N + 68), 7.0, device="cuda")
    aq.aq_lora_add(lora, Xd, idd, part, out=apart[1:-1, 4:4 + N])
    h = host(apart)
    assert np.array_equal(h[1:-1, 4:4 + N], ref) and np.array_equal(host(G), wide)
    h[1:-1, 4:4 + N] = 7
    assert (h == 7).all()
    aq.aq_lora_add(lora, Xd, idd, part, out=part)
    h, want = host(G), wide.copy()
    want[1:-1, 64:64 + N] = ref
    assert np.array_equal(h, want)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("f", [1e-30, 1e30])
def test_lora_tiles_small_and_large_values(t, f):
    """Values near the ends of FP32's range, in tiles.  A piece or a product below
    2^-126 may be taken for 0: a term of v is then off by 2^-126 (2 |a| + 12) more
    (two lower pieces; six products and their additions), one of Y likewise, which
    adds sum_r (|b| (scale e_v + 2^-125) + 12 2^-126), e_v = K 2^-126 (2 max |a| + 12),
    to the bound of the other tests."""
    K, N, L, R = 512, 576, 2, 128
    M = tokens_for_tiles(K, N, R, t)
    assert not by_rows(M, L, K, N, R, t)
    pool = [x.nan_to_num(0, 0, 0) if x.is_floating_point() else x for x in device_pool(9, L, R, K, N, t)]
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, L, M).astype(np.int32)
    X = gen.acts_outliers(rng, M, K, 5, 30.0) * np.float32(f)
    Y = rng.standard_normal((M, N)).astype(np.float32) * np.float32(f)
    say(f"  x{f} {t} M{M}")
    got = host(aq.aq_lora_add(aq.aq_lora_adapters(*pool), to_dev(X), to_dev(ids), to_dev(Y)))
    A, B, sc, ranks = (host(x).astype(np.float64) for x in pool)
    tiny = 2.0 ** -126
    for m in np.unique(np.r_[0, M - 1, rng.integers(0, M, 40)]):
        y, mag, low, a = Y[m].astype(np.float64), np.abs(Y[m].astype(np.float64)), 0.0, ids[m]
        if a >= 0:
            r = int(ranks[a])
            av, b = A[a, :r] * X[m].astype(np.float64), np.abs(B[a, :, :r])
            y = y + sc[a] * (B[a, :, :r] * av.sum(1)).sum(1)
            mag = mag + sc[a] * (b * np.abs(av).sum(1)).sum(1)
            ev = K * tiny * (2 * np.abs(A[a]).max() + 12)
            low = (b * (sc[a] * ev + 2 * tiny) + 12 * tiny).sum(1)
        assert (np.abs(got[m] - y) <= (K + R + 20) * 2.0 ** -24 * mag + low).all(), (m, a)
        assert np.linalg.norm(got[m] - y) <= 1e-5 * np.linalg.norm(y)
