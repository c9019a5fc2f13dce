"""The per-token-factor operators (router, mixture-of-experts layer over
packed experts, low-rank adapters) against their FP64 definitions.

Tolerances, from the arithmetic (u = 2^-24, half a step of FP32):
  * router: scores, choice and weights are formed in FP64 and rounded once,
    so ids are equal and a weight is off by u |w| (plus 2^-40 |w| for the
    FP64 sums, whose error is below 10^4 2^-53);
  * experts: gate and up sums are FP64 and h is rounded once, so the INT8
    codes of h equal the definition's; what is left are the FP32 sums of the
    down projection: C products and C - 1 additions of tile terms, the two
    scalings and top_k additions, (2C + top_k + 4) u of the sum of the terms'
    magnitudes;
  * adapters: FP32 products and sums over K, over the column ranges (at most
    64), over R, the scale and the last addition: (K + R + 80) u of the sum of
    the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
from oracle import aq_oracle as O
from oracle import routed as RO
from tests.parity import say, to_dev
from workloads import gen

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def host(t):
    torch.cuda.synchronize()
    return t.detach().cpu().float().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.detach().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()


# ---------------------------------------------------------------- router

def check_route(X, Wr, k, bias=None, score="softmax", norm=True, scale=1.0, name=""):
    Xd, Wd = to_dev(X), Wr.cuda() if isinstance(Wr, torch.Tensor) else to_dev(Wr)
    bd = None if bias is None else to_dev(bias)
    ids, w = aq.aq_moe_route(Xd, Wd, k, bias=bd, score=score, norm=norm, scale=scale)
    rid, rw = RO.route(X, host(Wd), k, bias, score, norm, float(np.float32(scale)))
    ids, w = host(ids), host(w).astype(np.float64)
    assert np.array_equal(ids, rid), f"{name}: {np.argwhere(ids != rid)[:4].tolist()}"
    err = np.abs(w - rw)
    say(f"  route {name}: worst weight error / |w| {float((err / np.maximum(np.abs(rw), 1e-300)).max()):.2e}")
    assert (err <= (U + 2.0 ** -40) * np.abs(rw) + 2.0 ** -149).all()
    return ids, w


@pytest.mark.parametrize("M,K,E,k,score,bias,norm,wtype", [
    (1, 2048, 128, 8, "softmax", False, True, "bf16"),
    (1, 64, 1, 1, "softmax", False, True, "f32"),
    (3, 128, 65, 32, "sigmoid", True, False, "f32"),
    (17, 4096, 250, 6, "sigmoid", True, True, "f32"),
    (33, 2560, 64, 1, "softmax", True, False, "bf16"),
    (130, 704, 1024, 8, "softmax", False, True, "f32"),
    (1024, 1024, 17, 17, "softmax", False, False, "bf16"),
])
def test_route(M, K, E, k, score, bias, norm, wtype):
    rng = np.random.default_rng(M * 7 + E)
    X = gen.acts_outliers(rng, M, K, max(1, K // 100), 30.0)
    W = (rng.standard_normal((E, K)) * 0.4 / np.sqrt(K)).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    check_route(X, bf16(W) if wtype == "bf16" else W, k, b, score, norm, 2.5 if norm else 1.0, f"M{M} E{E} k{k}")


def test_route_ties_and_exclusions():
    rng = np.random.default_rng(5)
    # whole numbers: every sum is exact, equal rows give equal keys
    X = rng.integers(-4, 5, (9, 128)).astype(np.float32)
    W = np.repeat(rng.integers(-2, 3, (5, 128)), 14, axis=0).astype(np.float32)[rng.permutation(70)]
    for score in ("softmax", "sigmoid"):
        check_route(X, W / 16, 9, None, score, True, name=f"ties {score}")
    check_route(np.zeros((2, 128), np.float32), W, 8, name="all equal")
    # a bias of -inf excludes; more slots than experts left; none left at all
    b = np.zeros(70, np.float32)
    b[rng.permutation(70)[:65]] = -np.inf
    for score in ("softmax", "sigmoid"):
        ids, w = check_route(X, W / 16, 9, b, score, True, name=f"five left {score}")
        assert (ids[:, 5:] == -1).all() and (w[:, 5:] == 0).all() and (ids[:, :5] >= 0).all()
        ids, w = check_route(X, W / 16, 9, np.full(70, -np.inf, np.float32), score, True, name="none left")
        assert (ids == -1).all() and (w == 0).all()


def test_route_far_logits():
    X = np.zeros((3, 64), np.float32)
    X[:, 0] = (1.0, 1000.0, -1000.0)
    W = np.zeros((6, 64), np.float32)
    W[:, 0] = (1, -1, 3, 2, -3, 0)
    for score in ("softmax", "sigmoid"):
        ids, w = check_route(X, W, 3, None, score, False, name=f"far {score}")
        assert np.isfinite(w).all()
    # with norm the weights of the chosen stay a distribution although their
    # shares of the whole softmax are below the smallest double
    b = np.array([0, 1e5, 0, 0, 1e5, 1e5], np.float32)
    _, w = check_route(X, W, 3, b, "softmax", True, name="far norm")
    assert np.abs(w.sum(1) - 1).max() < 1e-6


# ---------------------------------------------------------------- experts

class Experts:
    def __init__(self, E, H, I, frac8=0.3, bK=(128, 128), seed=0):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I, self.bK = E, H, I, bK
        W13, W2 = gen.weights(rng, E * 2 * I, H), gen.weights(rng, E * H, I)
        self.host = []
        pw = []
        for W, b in ((W13, bK[0]), (W2, bK[1])):
            z = gen.map_uniform(rng, W.shape[0] // 64, W.shape[1] // b, frac8)
            self.host.append(O.quant_weights(W, z, 64, b))
            pw.append(aq.aq_pack_weights(to_dev(W), aq.aq_labels_from_map(z.astype(np.uint8)), 64, b))
        self.dev = aq.PackedExperts(pw[0], pw[1], E)

    def check(self, X, ids, w, name="", rows=None):
        M, k = ids.shape
        qx, sx = aq.aq_quant_act(to_dev(X))
        Y = aq.aq_moe_experts(self.dev, qx, sx, to_dev(ids.astype(np.int32)), to_dev(w.astype(np.float32)))
        rows = np.arange(M) if rows is None else rows
        q, s = O.quant_act(X[rows])
        ref, mag = RO.experts(q, s, ids[rows], w[rows], self.host[0], self.host[1], self.E, self.bK)
        Y = host(Y)
        assert np.isfinite(Y).all()
        err = np.abs(Y[rows].astype(np.float64) - ref)
        tol = (2 * (self.I // self.bK[1]) + k + 4) * U * mag + 1e-30
        say(f"  experts {name}: worst error / bound {float((err / tol).max()):.3f}")
        assert (err <= tol).all(), np.argwhere(err > tol)[:4].tolist()
        return Y


def draws(rng, M, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32)
    w = rng.random((M, k)).astype(np.float32)
    return ids, w / w.sum(1, keepdims=True)


@pytest.mark.parametrize("M,E,k,H,I,frac8,bK", [
    (1, 8, 2, 256, 128, 0.3, (128, 128)),
    (1, 16, 8, 512, 384, 0.25, (128, 128)),
    (2, 1, 1, 128, 128, 0.0, (128, 128)),
    (5, 6, 3, 384, 320, 1.0, (128, 64)),
    (4, 5, 4, 192, 256, 0.5, (64, 128)),
    (16, 4, 2, 320, 192, 0.4, (64, 64)),
    (33, 12, 4, 640, 256, 0.3, (128, 128)),
    (70, 3, 2, 256, 512, 0.3, (128, 128)),
    (9, 40, 5, 2560, 128, 0.3, (128, 128)),
    (3, 2, 2, 128, 2560, 0.3, (128, 128)),
    # more tile columns than one window of labels holds, in either projection
    (4, 3, 2, 4160, 128, 0.4, (64, 64)),
    (19, 3, 2, 4160, 128, 0.4, (64, 128)),
    (4, 3, 2, 128, 4160, 0.4, (128, 64)),
    (20, 3, 3, 128, 4160, 0.4, (128, 64)),
    # column ranges of gate/up: 8 (more than there are tile columns, and not
    # dividing them), 4, 2, 1; pairs found by scan, then from lists
    (20, 32, 4, 128, 128, 0.3, (128, 128)),
    (64, 128, 8, 640, 64, 0.3, (128, 64)),
    (64, 128, 8, 384, 128, 0.3, (128, 128)),
    (64, 128, 8, 384, 256, 0.3, (128, 128)),
    (64, 128, 8, 192, 320, 0.3, (64, 64)),
    (130, 128, 4, 640, 64, 0.3, (128, 64)),
    (130, 128, 4, 384, 128, 0.3, (128, 128)),
    (130, 128, 4, 384, 256, 0.3, (128, 128)),
    (130, 128, 4, 192, 320, 0.3, (64, 64)),
    # down: several tile rows a walk, the last walk shorter
    (32, 64, 4, 2112, 64, 0.3, (64, 64)),
    (64, 128, 2, 2112, 64, 0.3, (64, 64)),
    (200, 128, 4, 2112, 64, 0.3, (64, 64)),
    # down: the longest rows that LDS holds, copied and quantized there, 32 a pass
    (40, 4, 2, 128, 2048, 0.3, (128, 128)),
    (30, 10, 2, 128, 2048, 0.3, (64, 64)),
    # whole rows per wave in gate/up, more and fewer than 16 tokens an expert,
    # columns that end inside a chunk, by scan and from lists
    (102, 33, 5, 640, 1024, 0.3, (128, 128)),
    (140, 33, 5, 640, 1024, 0.3, (128, 128)),
    (300, 128, 8, 192, 320, 0.3, (64, 64)),
    # an expert's passes side by side: more and fewer than its workgroups, each
    # number of column ranges, codes in LDS and not
    (250, 1, 1, 640, 128, 0.3, (128, 128)),
    (300, 4, 2, 384, 1024, 0.3, (128, 128)),
    (200, 3, 2, 192, 2112, 0.3, (64, 64)),
    (90, 2, 2, 512, 256, 0.3, (128, 64)),
])
def test_experts(M, E, k, H, I, frac8, bK):
    rng = np.random.default_rng(100 + M + E)
    ex = Experts(E, H, I, frac8, bK, seed=M)
    X = gen.acts_outliers(rng, M, H, max(1, H // 100), 30.0)
    ids, w = draws(rng, M, E, k)
    ex.check(X, ids, w, f"M{M} E{E} k{k} {H}x{I} bK{bK}")


def test_experts_odd_ids():
    """Slots without an expert, tokens without any, the same expert twice in a
    row, every token at one expert, expert ids far outside."""
    rng = np.random.default_rng(9)
    ex = Experts(7, 256, 256, seed=3)
    for M in (1, 4, 37):
        X = gen.acts_outliers(rng, M, 256, 2, 30.0)
        ids, w = draws(rng, M, 7, 4)
        ids[rng.random(ids.shape) < 0.4] = -1
        ids[0, 1] = 7
        ids[-1, 0] = np.iinfo(np.int32).min
        ids[M // 2] = (3, 3, 3, 1 << 30)
        Y = ex.check(X, ids, w, f"odd ids M{M}")
        Y = ex.check(X, np.full_like(ids, 5), w, f"one expert M{M}")
        Y = ex.check(X, np.full_like(ids, -1), w, f"no expert M{M}")
        assert (Y == 0).all()


def test_experts_odd_values():
    """Zero tokens (all codes 0), gates far below and above zero (h underflows
    to 0 or is g * u), zero and negative weights."""
    rng = np.random.default_rng(10)
    ex = Experts(3, 128, 128, seed=4)
    X = gen.acts_outliers(rng, 6, 128, 2, 30.0)
    X[1] = 0
    X[2] *= 1e4
    X[3] *= 1e-20
    X[4] *= 1e6
    ids, w = draws(rng, 6, 3, 3)
    w[5] = (0.0, -1.5, 2.0)
    Y = ex.check(X, ids, w, "odd values")
    assert (Y[1] == 0).all()


def test_pack_experts():
    """The layer's packing helper puts every expert's rows where the calls look
    for them."""
    from mixed_precision_int_amd.model import pack_experts
    E, H, I = 3, 256, 128
    ex = Experts(E, H, I, seed=12)
    rng = np.random.default_rng(12)
    W13, W2 = gen.weights(rng, E * 2 * I, H), gen.weights(rng, E * H, I)
    z13 = gen.map_uniform(np.random.default_rng(1), E * 2 * I // 64, H // 128, 0.4)
    z2 = gen.map_uniform(np.random.default_rng(2), E * H // 64, I // 128, 0.4)
    W = to_dev(W13).view(E, 2 * I, H)
    ex.dev = pack_experts(W[:, :I].contiguous(), W[:, I:].contiguous(), to_dev(W2).view(E, H, I), z13, z2)
    ex.host = [O.quant_weights(W13, z13, 64, 128), O.quant_weights(W2, z2, 64, 128)]
    assert (ex.dev.H, ex.dev.I, ex.dev.E) == (H, I, E)
    ids, w = draws(rng, 5, E, 2)
    ex.check(gen.acts_outliers(rng, 5, H, 2, 30.0), ids, w, "pack_experts")


@pytest.mark.parametrize("M", [256, 1024])
def test_experts_many_tokens(M):
    rng = np.random.default_rng(M)
    ex = Experts(5, 256, 192, seed=6, bK=(128, 64))
    X = gen.acts_outliers(rng, M, 256, 2, 30.0)
    ids, w = draws(rng, M, 5, 2)
    ids[: M // 2] = (0, 4)                   # one expert holds half of the tokens
    ex.check(X, ids, w, f"M{M}", rows=np.unique(rng.integers(0, M, 24)))


@pytest.mark.parametrize("M,E,k", [(130, 128, 4), (200, 300, 4), (300, 60, 2)])
def test_experts_skewed(M, E, k):
    """Many pairs over many experts, a third of the tokens at the same ones,
    some slots without an expert, most experts without a pair."""
    rng = np.random.default_rng(M + 1)
    ex = Experts(E, 256, 128, seed=7)
    X = gen.acts_outliers(rng, M, 256, 2, 30.0)
    ids, w = draws(rng, M, E, k)
    ids[rng.random(M) < 0.33] = np.arange(k) + E - k
    ids[ids > 9] = np.where(rng.random((ids > 9).sum()) < 0.5, ids[ids > 9], -1)
    ex.check(X, ids, w, f"skewed M{M}", rows=np.unique(rng.integers(0, M, 40)))


@pytest.mark.parametrize("M", [1025, 2500])
def test_experts_long_batches(M):
    """Longer batches take the tokens 1024 at a time: a pass gives what a call
    for its tokens gives, bit for bit."""
    rng = np.random.default_rng(M)
    ex = Experts(9, 256, 192, seed=6, bK=(128, 64))
    Xd = to_dev(gen.acts_outliers(rng, M, 256, 2, 30.0))
    Wr = to_dev((rng.standard_normal((9, 256)) * 0.05).astype(np.float32))
    Y, ids, w = aq.aq_moe_layer(ex.dev, Xd, Wr, 3)
    i2, w2 = aq.aq_moe_route(Xd, Wr, 3)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    qx, sx = aq.aq_quant_act(Xd)
    assert torch.equal(aq.aq_moe_experts(ex.dev, qx, sx, ids, w), Y)
    ex.check(host(Xd), host(ids), host(w), f"M{M}", rows=np.unique(np.r_[rng.integers(0, M, 12), 1023, 1024, M - 1]))
    for m in range(0, M, 1024):
        s = slice(m, m + 1024)
        y = aq.aq_moe_experts(ex.dev, qx[s].contiguous(), sx[s].contiguous(), ids[s].contiguous(), w[s].contiguous())
        assert torch.equal(y, Y[s])


def test_experts_past_32_bits():
    """Packed weights of more than 2^31 bytes: the last expert's outputs are
    those of the same expert packed alone.  Bit for bit, although the column
    ranges of gate/up differ between the two: every tile row holds 127 / 1024, so
    that the W8 scale is 2^-10 and the W4 scale one FP32 constant below 2^-5, and
    the FP64 sums (32 products below 2^21 times a multiple of 2^-30) are exact."""
    E, H, I = 66, 4096, 4096
    gen_ = torch.Generator(device="cuda").manual_seed(3)
    g = torch.zeros((E, 2 * I, H), device="cuda")
    d = torch.zeros((E, H, I), device="cuda")
    for t in (g, d):
        t[-1] = torch.randint(-127, 128, t[-1].shape, device="cuda", generator=gen_).float() / 1024
        t[-1, :, ::128] = 127 / 1024

    def pack(g, d):
        n = len(g)
        out = []
        for W in (g.view(-1, H), d.view(-1, I)):
            z = np.full((W.shape[0] // 64, W.shape[1] // 128), 8, np.uint8)
            z[-1, ::2] = 4
            out.append(aq.aq_pack_weights(W, aq.aq_labels_from_map(z), 64, 128))
        return aq.PackedExperts(out[0], out[1], n)
    many, one = pack(g, d), pack(g[-1:].contiguous(), d[-1:].contiguous())
    del g, d
    assert many.gate_up.plan.w8_bytes > 1 << 31
    for M in (1, 9, 40, 600):
        X = torch.randn((M, H), device="cuda", generator=gen_)
        qx, sx = aq.aq_quant_act(X)
        ids = torch.full((M, 1), E - 1, dtype=torch.int32, device="cuda")
        w = torch.rand((M, 1), device="cuda", generator=gen_)
        say(f"  past 32 bits, M{M}")
        a = aq.aq_moe_experts(many, qx, sx, ids, w)
        b = aq.aq_moe_experts(one, qx, sx, torch.zeros_like(ids), w)
        assert torch.equal(a, b) and bool((a != 0).any())


@pytest.mark.parametrize("M", [1, 3, 8, 20, 65])
def test_layer_is_its_parts(M):
    """aq_moe_layer equals aq_quant_act, aq_moe_route and aq_moe_experts bit
    for bit, and the definition."""
    rng = np.random.default_rng(M)
    ex = Experts(11, 512, 256, seed=8)
    X = gen.acts_outliers(rng, M, 512, 5, 30.0)
    Wr = bf16(rng.standard_normal((11, 512)) * 0.02)
    b = to_dev((rng.standard_normal(11) * 0.1).astype(np.float32))
    b[2] = -float("inf")
    Xd = to_dev(X)
    Y, ids, w = aq.aq_moe_layer(ex.dev, Xd, Wr.cuda(), 3, bias=b, score="sigmoid", scale=1.5)
    qx, sx = aq.aq_quant_act(Xd)
    i2, w2 = aq.aq_moe_route(Xd, Wr.cuda(), 3, bias=b, score="sigmoid", scale=1.5)
    Y2 = aq.aq_moe_experts(ex.dev, qx, sx, i2, w2)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    assert torch.equal(Y.view(torch.int32), Y2.view(torch.int32))
    check_route(X, Wr, 3, host(b), "sigmoid", True, 1.5, f"layer M{M}")
    Y3 = ex.check(X, host(ids), host(w), f"layer M{M}")
    assert np.array_equal(host(Y), Y3)


@pytest.mark.parametrize("M,E,k,score", [
    (1, 100, 8, "softmax"), (5, 200, 4, "sigmoid"), (8, 256, 8, "softmax"), (3, 300, 2, "sigmoid"), (2, 1024, 5, "softmax"),
    (9, 128, 8, "sigmoid"), (40, 128, 6, "softmax"), (200, 70, 7, "sigmoid"),
])
def test_layer_many_experts(M, E, k, score):
    """The choice inside gate/up for more experts than lanes, beside the layer's
    other ways, with excluded experts and equal keys."""
    rng = np.random.default_rng(M + E)
    ex = Experts(E, 512, 64, seed=8, bK=(128, 64))
    X = rng.integers(-4, 5, (M, 512)).astype(np.float32)   # whole numbers: exact sums
    W = rng.integers(-2, 3, (E, 512)).astype(np.float32) / 256
    W[E // 2:] = W[: E - E // 2]                       # every expert twice: equal logits
    b = (rng.standard_normal(E // 2) * 0.1).astype(np.float32)
    b = np.r_[b, b, np.zeros(E % 2, np.float32)].astype(np.float32)
    b[rng.permutation(E)[: E - k + 1]] = -np.inf       # one slot too many
    for bias in (None, b):
        bd = None if bias is None else to_dev(bias)
        Y, ids, w = aq.aq_moe_layer(ex.dev, to_dev(X), to_dev(W), k, bias=bd, score=score)
        rid, _ = check_route(X, W, k, bias, score, name=f"layer M{M} E{E}")
        assert np.array_equal(host(ids), rid)
        qx, sx = aq.aq_quant_act(to_dev(X))
        assert torch.equal(Y, aq.aq_moe_experts(ex.dev, qx, sx, ids, w))
        rows = np.unique(rng.integers(0, M, 20))
        assert np.array_equal(ex.check(X, host(ids), host(w), f"layer M{M} E{E}", rows=rows), host(Y))


# ---------------------------------------------------------------- adapters

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def lora_case(rng, M, K, N, L, R, t, ranks=None, ids=None):
    A = torch.from_numpy((rng.standard_normal((L, R, K)) / np.sqrt(K)).astype(np.float32)).to(TYPES[t]).cuda()
    B = torch.from_numpy((rng.standard_normal((L, N, R)) * 0.1).astype(np.float32)).to(TYPES[t]).cuda()
    sc = (rng.random(L) + 0.5).astype(np.float32)
    if ranks is None:
        ranks = rng.integers(0, R + 1, L)
    if ids is None:
        ids = rng.integers(-1, L, M)
    X = gen.acts_outliers(rng, M, K, max(1, K // 100), 30.0)
    Y = rng.standard_normal((M, N)).astype(np.float32)
    return A, B, sc, ranks.astype(np.int32), ids.astype(np.int32), X, Y


def check_lora(A, B, sc, ranks, ids, X, Y, name="", rows=None, out=None):
    ad = aq.aq_lora_adapters(A, B, None if sc is None else to_dev(sc), None if ranks is None else to_dev(ranks))
    got = aq.aq_lora_add(ad, to_dev(X), to_dev(ids), to_dev(Y), out=out)
    rows = np.arange(len(ids)) if rows is None else rows
    ref, mag = RO.lora(Y[rows], X[rows], ids[rows], host(A), host(B), sc, ranks)
    got = host(got)
    err = np.abs(got[rows].astype(np.float64) - ref)
    tol = (X.shape[1] + A.shape[1] + 80) * U * mag + 1e-30
    say(f"  lora {name}: worst error / bound {float((err / tol).max()):.4f}, normwise {np.linalg.norm(err) / np.linalg.norm(ref):.2e}")
    assert (err <= tol).all(), np.argwhere(~(err <= tol))[:4].tolist()
    # the FP32 sums' errors are independent: far below the worst case
    assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(ref)
    none = (ids < 0) | (ids >= A.shape[0])
    assert np.array_equal(got[none], Y[none])
    return got


@pytest.mark.parametrize("M,K,N,L,R,t", [
    (1, 4096, 512, 3, 16, "bf16"),
    (1, 64, 64, 1, 8, "f32"),
    (7, 2560, 320, 4, 8, "f16"),
    (16, 1024, 1024, 20, 32, "bf16"),
    (33, 704, 192, 2, 128, "f32"),
    (64, 1024, 448, 64, 64, "f16"),
    (90, 512, 256, 5, 24, "bf16"),
    (333, 320, 640, 6, 16, "f32"),
    (1030, 192, 128, 7, 40, "bf16"),
    (257, 1088, 320, 3, 128, "f32"),
    (300, 64, 64, 40, 128, "f16"),
    (520, 2048, 96 * 2, 2, 64, "f32"),
    (700, 640, 192, 3, 8, "f16"),
    (1500, 1024, 2048, 3, 64, "f32"),
    (260, 4096, 2048, 2, 128, "bf16"),
    (640, 2048, 2048, 40, 64, "bf16"),
    (4100, 1024, 1088, 5, 16, "f16"),
])
def test_lora(M, K, N, L, R, t):
    rng = np.random.default_rng(M + R)
    c = lora_case(rng, M, K, N, L, R, t)
    check_lora(*c, name=f"M{M} {N}x{K} L{L} R{R} {t}")
    # the same tokens in runs, as prompts one after another
    check_lora(*c[:4], np.sort(c[4]), *c[5:], name="runs")
    check_lora(*c[:4], np.full(M, L - 1, np.int32), *c[5:], name="one")


@pytest.mark.parametrize("M", [1, 40, 200, 500])
def test_lora_isolation(M):
    """What lies beyond an adapter's rank, another request's adapter and
    another request's activations never enter a token's result."""
    rng = np.random.default_rng(17)
    A, B, sc, ranks, ids, X, Y = lora_case(rng, M, 256, 192, 4, 16, "bf16", ranks=np.array([5, 16, 0, 11]))
    ids[:] = rng.integers(-1, 3, M)
    want = check_lora(A, B, sc, ranks, ids, X, Y, "clean")
    for a, r in enumerate(ranks):
        A[a, r:] = float("nan")
        B[a, :, r:] = float("inf")
    A[3], B[3] = float("inf"), float("nan")   # no token of this call has it
    got = check_lora(A, B, sc, ranks, ids, X, Y, "padding")
    assert np.array_equal(got, want)
    if M > 1:
        ids2, X2 = ids.copy(), X.copy()
        ids2[M // 2], X2[M // 3] = 3, np.nan
        ad = aq.aq_lora_adapters(A, B, to_dev(sc), to_dev(ranks))
        got = host(aq.aq_lora_add(ad, to_dev(X2), to_dev(ids2), to_dev(Y)))
        keep = np.ones(M, bool)
        keep[[M // 2, M // 3]] = False
        assert np.array_equal(got[keep], want[keep])


@pytest.mark.parametrize("M", [1, 5, 100, 330])
def test_lora_slices_and_in_place(M):
    """A member's columns of a grouped output, in place and into a contiguous
    tensor; the columns beside it stay as they were."""
    rng = np.random.default_rng(M)
    A, B, sc, ranks, ids, X, _ = lora_case(rng, M, 256, 128, 3, 8, "f16", ranks=np.array([8, 3, 8]))
    wide = rng.standard_normal((M, 448)).astype(np.float32)
    ad = aq.aq_lora_adapters(A, B, to_dev(sc), to_dev(ranks))
    G = to_dev(wide)
    ref = check_lora(A, B, sc, ranks, ids, X, wide[:, 192:320].copy(), "slice")
    apart = aq.aq_lora_add(ad, to_dev(X), to_dev(ids), G[:, 192:320])
    assert np.array_equal(host(apart), ref) and np.array_equal(host(G), wide)
    res = aq.aq_lora_add(ad, to_dev(X), to_dev(ids), G[:, 192:320], out=G[:, 192:320])
    got = host(G)
    assert res.data_ptr() == G[:, 192:320].data_ptr()
    assert np.array_equal(got[:, 192:320], ref)
    assert np.array_equal(got[:, :192], wide[:, :192]) and np.array_equal(got[:, 320:], wide[:, 320:])


@pytest.mark.parametrize("M,L", [(9000, 3), (20000, 1000), (3000, 8192)])
def test_lora_many_tokens_and_adapters(M, L):
    """More tokens than the grouping keeps in registers, and adapter pools up to
    the largest; some rows against the definition, all against a second call
    with the tokens in another order."""
    rng = np.random.default_rng(L)
    A, B, sc, ranks, ids, X, Y = lora_case(rng, M, 128, 1024, L, 8, "bf16")
    got = check_lora(A, B, sc, ranks, ids, X, Y, f"M{M} L{L}", rows=np.unique(rng.integers(0, M, 60)))
    perm = rng.permutation(M)
    again = check_lora(A, B, sc, ranks, ids[perm], X[perm], Y[perm], "permuted", rows=np.arange(10))
    assert np.array_equal(again, got[perm])


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R", [8, 16, 24, 40, 64, 72, 128])
def test_lora_tiles(R, t):
    """Enough tokens to be grouped (128 MiB of adapter rows), most of them at one
    adapter, a few tokens at others, some ranks cut, NaN beyond them."""
    K, N, L = 1088, 1152, 6
    rng = np.random.default_rng(R)
    M = (128 << 20) // (R * (K + N) * (4 if t == "f32" else 2)) + 5
    ids = np.where(rng.random(M) < 0.9, 1, rng.integers(-1, L, M))
    ids[ids == 4] = 1
    ids[[3, M - 2]] = 4                      # an adapter with two tokens
    ranks = np.array([R, R, max(R - 5, 1), 0, R // 2 + 1, R])
    A, B, sc, ranks, ids, X, Y = lora_case(rng, M, K, N, L, R, t, ranks=ranks, ids=ids)
    for a in range(L):
        A[a, ranks[a]:] = float("nan")
        B[a, :, ranks[a]:] = float("nan")
    rows = np.unique(np.r_[3, M - 2, rng.integers(0, M, 40), np.flatnonzero(ids == 2)[:4], np.flatnonzero(ids == -1)[:2]])
    check_lora(A, B, sc, ranks, ids, X, Y, f"tiles R{R} {t} M{M}", rows=rows)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_lora_small_and_large_values(t):
    """Values whose smallest pieces lie near the ends of FP32's range."""
    rng = np.random.default_rng(8)
    for M in (9, 700):
        for fx, fy in ((1e-30, 1e-30), (1e30, 1e30)):
            A, B, sc, ranks, ids, X, Y = lora_case(rng, M, 512, 192, 2, 128, t)
            check_lora(A, B, sc, ranks, ids, X * np.float32(fx), Y * np.float32(fy), f"x{fx} M{M} {t}")


@pytest.mark.parametrize("M,L", [(64, 64), (63, 9), (17, 1), (65, 3)])
def test_lora_tokens_alone(M, L):
    """Among a few tokens the result of each is the one it has alone, bit for bit."""
    rng = np.random.default_rng(M)
    A, B, sc, ranks, ids, X, Y = lora_case(rng, M, 320, 256, L, 24, "bf16")
    out = check_lora(A, B, sc, ranks, ids, X, Y, f"alone M{M} L{L}")
    lora = aq.aq_lora_adapters(A, B, to_dev(sc), to_dev(ranks))
    for m in range(0, M, 5):
        one = aq.aq_lora_add(lora, to_dev(X[m:m + 1]), to_dev(ids[m:m + 1]), to_dev(Y[m:m + 1]))
        assert np.array_equal(host(one)[0], out[m])


@pytest.mark.parametrize("K,N,R", [(4096, 64, 8), (64, 4096, 24)])
def test_lora_past_32_bits(K, N, R):
    """X or Y of more than 2^31 elements."""
    M, L = (1 << 19) + 77, 3
    g = torch.Generator(device="cuda").manual_seed(K)
    A = torch.randn((L, R, K), device="cuda", generator=g)
    B = torch.randn((L, N, R), device="cuda", generator=g)
    X = torch.randn((M, K), device="cuda", generator=g)
    Y = torch.randn((M, N), device="cuda", generator=g)
    ids = torch.randint(-1, L, (M,), device="cuda", generator=g, dtype=torch.int32)
    rows = torch.tensor([0, 1, M // 2, M - 78, M - 2, M - 1], device="cuda")
    y0, x0 = Y[rows], X[rows]
    say(f"  lora M{M} K{K} N{N}")
    aq.aq_lora_add(aq.aq_lora_adapters(A, B), X, ids, Y, out=Y)
    ref, mag = RO.lora(host(y0).astype(np.float64), host(x0), host(ids[rows]), host(A), host(B))
    err = np.abs(host(Y[rows]).astype(np.float64) - ref)
    assert (err <= (K + R + 80) * U * mag).all()


def test_lora_tiles_replayed():
    """The grouped form captured, on two streams, and replayed between eager
    calls: every result equals the eager one's."""
    rng = np.random.default_rng(31)
    M, K, N, L, R = 450, 512, 576, 4, 128
    A, B, sc, ranks, ids, X, Y = lora_case(rng, M, K, N, L, R, "f32")
    lora = aq.aq_lora_adapters(A, B, to_dev(sc), to_dev(ranks))
    Xd, Yd, idd = to_dev(X), to_dev(Y), to_dev(ids)
    aq.aq_lora_add(lora, Xd, idd, Yd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = aq.aq_lora_add(lora, Xd, idd, Yd)
    side = torch.cuda.Stream()
    for _ in range(4):
        idd.copy_(to_dev(rng.integers(-1, L + 1, M).astype(np.int32)))
        Xd.copy_(to_dev(gen.acts_outliers(rng, M, K, 5, 30.0)))
        want = aq.aq_lora_add(lora, Xd, idd, Yd)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        other = aq.aq_lora_add(lora, Xd, idd, Yd, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)


def test_lora_most_rows():
    """The longest batch that is taken by rows (below 128 MiB of adapter rows)."""
    rng = np.random.default_rng(77)
    c = lora_case(rng, 65535, 64, 64, 4, 8, "bf16")
    check_lora(*c, name="rows 65535", rows=np.unique(np.r_[0, 65534, rng.integers(0, 65535, 60)]))


def test_no_tokens():
    """Calls without tokens do nothing and return empty outputs."""
    _, _, lora, _, ex, Wr, _, _ = _system(3, seed=6)
    X = torch.empty((0, 512), device="cuda")
    e, w = aq.aq_moe_route(X, Wr, 4)
    assert e.shape == w.shape == (0, 4)
    Y, e, w = aq.aq_moe_layer(ex.dev, X, Wr, 4)
    assert Y.shape == (0, 512) and e.shape == (0, 4)
    qx, sx = torch.empty((0, 512), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    assert aq.aq_moe_experts(ex.dev, qx, sx, e, w).shape == (0, 512)
    assert aq.aq_lora_add(lora, X, torch.empty(0, dtype=torch.int32, device="cuda"), X).shape == (0, 512)


@pytest.mark.parametrize("M", [3, 40, 1100])
def test_padded_batch(M):
    """Rows of a padded batch that hold NaN and infinities change nothing for the
    others, in any of the calls, and every id stays in range."""
    _, _, lora, _, ex, Wr, X, ids = _system(M, seed=7)
    bad = np.arange(0, M, 3)
    Xb = X.copy()
    Xb[bad[::2]] = np.nan
    Xb[bad[1::2]] = np.inf
    Xb[bad, ::2] *= -1
    idd = to_dev(ids)
    good = torch.from_numpy(np.setdiff1d(np.arange(M), bad)).cuda()
    out = []
    for x in (to_dev(X), to_dev(Xb)):
        y = aq.aq_lora_add(lora, x, idd, x)
        Z, e, w = aq.aq_moe_layer(ex.dev, x, Wr, 4)
        assert bool(((e >= -1) & (e < 12)).all())
        out.append([t[good] for t in (y, Z, e, w)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_lora_defaults_and_ids_outside():
    rng = np.random.default_rng(3)
    A, B, _, _, _, X, Y = lora_case(rng, 6, 128, 64, 2, 8, "f32")
    ids = np.array([0, 1, 2, -7, 1 << 30, 1], np.int32)
    check_lora(A, B, None, None, ids, X, Y, "defaults")
    check_lora(A, B, None, np.array([100, -3], np.int32), ids, X, Y, "clamped ranks")
    check_lora(A, B, None, None, np.full(6, -1, np.int32), X, Y, "no adapter")


# ---------------------------------------------------------------- together

def _step(pw, lora, experts, Wr, X, ids, bias=None):
    """A layer's worth as a serving loop calls it: a shared projection with
    the requests' adapters beside it, then the experts."""
    qx, sx = aq.aq_quant_act(X)
    Y = aq.aq_linear_decode(pw, qx, sx)
    aq.aq_lora_add(lora, X, ids, Y, out=Y)
    Z, e, w = aq.aq_moe_layer(experts, Y, Wr, 4, bias=bias)
    return Y, Z, e, w


def _system(M, seed=0):
    rng = np.random.default_rng(seed)
    H = 512
    W = gen.weights(rng, H, H)
    z = gen.map_uniform(rng, H // 64, H // 128, 0.3)
    pw = aq.aq_pack_weights(to_dev(W), aq.aq_labels_from_map(z.astype(np.uint8)))
    A, B, sc, ranks, ids, X, _ = lora_case(rng, M, H, H, 5, 16, "bf16")
    ex = Experts(12, H, 256, seed=seed)
    Wr = to_dev((rng.standard_normal((12, H)) * 0.02).astype(np.float32))
    return pw, (W, z), aq.aq_lora_adapters(A, B, to_dev(sc), to_dev(ranks)), (A, B, sc, ranks), ex, Wr, X, ids


@pytest.mark.parametrize("M", [1, 6, 40])
def test_run_together(M):
    pw, (W, z), lora, (A, B, sc, ranks), ex, Wr, X, ids = _system(M)
    Y, Z, e, w = _step(pw, lora, ex.dev, Wr, to_dev(X), to_dev(ids))
    # adapters over the shared projection
    q, s = O.quant_act(X)
    codes, sW = O.quant_weights(W, z, 64, 128)
    base, mag0 = RO.linear64(q, s, codes, sW, 128)
    ref, mag = RO.lora(base, X, ids, host(A), host(B), sc, ranks)
    err = np.abs(host(Y).astype(np.float64) - ref)
    assert (err <= (512 + 16 + 80) * U * (mag + mag0)).all()
    # the experts over what the kernels produced
    Yh = host(Y)
    check_route(Yh, host(Wr), 4, name="together")
    got = ex.check(Yh, host(e), host(w), "together")
    assert np.array_equal(got, host(Z))


@pytest.mark.parametrize("M", [1, 7, 70, 200])
def test_graph_replay(M):
    """Captured and replayed with new inputs between eager calls: every replay
    equals the eager run."""
    pw, _, lora, _, ex, Wr, X, ids = _system(M, seed=1)
    rng = np.random.default_rng(4)
    Xd, idd = to_dev(X), to_dev(ids)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        _step(pw, lora, ex.dev, Wr, Xd, idd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(pw, lora, ex.dev, Wr, Xd, idd)
    for _ in range(4):
        Xd.copy_(to_dev(gen.acts_outliers(rng, M, 512, 5, 30.0)))
        idd.copy_(to_dev(rng.integers(-1, 5, M).astype(np.int32)))
        want = [t.clone() for t in _step(pw, lora, ex.dev, Wr, Xd, idd)]
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_two_streams():
    """Calls on two streams at once, each with its own workspace."""
    pw, _, lora, _, ex, Wr, X, ids = _system(24, seed=2)
    Xs = [to_dev(X), to_dev(X[::-1].copy())]
    idd = to_dev(ids)
    want = []
    for x in Xs:
        y = aq.aq_lora_add(lora, x, idd, x)
        want.append((y, *aq.aq_moe_layer(ex.dev, y, Wr, 4)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for x, st in zip(Xs, streams):
            y = aq.aq_lora_add(lora, x, idd, x, stream=st)
            got.append((y, *aq.aq_moe_layer(ex.dev, y, Wr, 4, stream=st)))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_refused_tensors():
    """What the binding refuses before any call: other types, shapes, layouts."""
    pw, _, lora, _, ex, Wr, X, ids = _system(5, seed=5)
    Xd, idd = to_dev(X), to_dev(ids)
    qx, sx = aq.aq_quant_act(Xd)
    e, w = aq.aq_moe_route(Xd, Wr, 4)
    bad = [
        lambda: aq.aq_moe_route(Xd.double(), Wr, 4), lambda: aq.aq_moe_route(Xd, Wr.half(), 4),
        lambda: aq.aq_moe_route(Xd, Wr[:, :256].contiguous(), 4), lambda: aq.aq_moe_route(Xd.t(), Wr, 4),
        lambda: aq.aq_moe_route(Xd, Wr, 4, bias=Wr[0]), lambda: aq.aq_moe_route(Xd, Wr, 4, score="topk"),
        lambda: aq.aq_moe_route(Xd, Wr, 4, ids=e.long()), lambda: aq.aq_moe_route(Xd.cpu(), Wr, 4),
        lambda: aq.aq_moe_route(Xd, Wr.cpu(), 4),
        lambda: aq.aq_moe_experts(ex.dev, qx, sx, e.long(), w), lambda: aq.aq_moe_experts(ex.dev, qx, sx[:3], e, w),
        lambda: aq.aq_moe_experts(ex.dev, qx, sx, e, w[:, :2]), lambda: aq.aq_moe_experts(ex.dev, qx[:, :256], sx, e, w),
        lambda: aq.aq_moe_layer(ex.dev, Xd, Wr, 4, ws=torch.empty(1 << 24, dtype=torch.uint8)),
        lambda: aq.aq_moe_layer(ex.dev, Xd, Wr[:8].contiguous(), 4), lambda: aq.aq_moe_layer(ex.dev, Xd, Wr, 4, out=Xd.half()),
        lambda: aq.aq_lora_add(lora, Xd, idd.long(), Xd), lambda: aq.aq_lora_add(lora, Xd, idd, Xd[:, :256]),
        lambda: aq.aq_lora_add(lora, Xd, idd, Xd.t().contiguous().t()), lambda: aq.aq_lora_add(lora, Xd, idd[:2], Xd),
        lambda: aq.aq_lora_adapters(lora.A, lora.B.float()), lambda: aq.aq_lora_adapters(lora.A.int(), lora.B.int()),
        lambda: aq.aq_lora_adapters(lora.A, lora.B, ranks=idd[:4]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            say(f"  call {i} was taken")
    # and the library: more experts a token than there are, too many tokens, a
    # workspace that is too small, an output that overlaps the input
    for f, status in [
        (lambda: aq.aq_moe_route(Xd, Wr, 13), -8), (lambda: aq.aq_moe_route(Xd, Wr, 0), -8),
        (lambda: aq.aq_moe_route(Xd, Wr, 4, scale=float("nan")), -8),
        (lambda: aq.aq_moe_layer(ex.dev, Xd, Wr, 4, ws=torch.empty(1024, dtype=torch.uint8, device="cuda")), -6),
        (lambda: aq.aq_lora_add(lora, Xd, idd, Xd, ws=torch.empty(16, dtype=torch.uint8, device="cuda")), -6),
    ]:
        with pytest.raises(aq.AqError) as err:
            f()
        assert err.value.status == status
    big = torch.zeros((6, 512), device="cuda")
    with pytest.raises(aq.AqError) as err:
        aq.aq_lora_add(lora, Xd, idd, big[:5], out=big[1:])
    assert err.value.status == -8


def test_given_outputs_and_workspace():
    pw, _, lora, _, ex, Wr, X, ids = _system(5, seed=3)
    Xd = to_dev(X)
    Y, e, w = aq.aq_moe_layer(ex.dev, Xd, Wr, 4)
    ws = torch.full((aq.aq_moe_workspace_bytes(ex.dev, 5, 4),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(Y, float("nan"))
    e2, w2 = torch.full_like(e, -9), torch.full_like(w, float("nan"))
    r = aq.aq_moe_layer(ex.dev, Xd, Wr, 4, out=out, ids=e2, weights=w2, ws=ws)
    assert r[0] is out and torch.equal(out, Y) and torch.equal(e2, e) and torch.equal(w2, w)
    empty = aq.aq_moe_layer(ex.dev, Xd[:0], Wr, 4)
    assert empty[0].shape == (0, 512) and empty[1].shape == (0, 4)
    assert aq.aq_lora_add(lora, Xd[:0], to_dev(ids[:0]), Xd[:0]).shape == (0, 512)
