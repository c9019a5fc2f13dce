"""A decoder layer's steps between its projections against their FP64
definitions (oracle/layer.py).

Tolerances, from the arithmetic (u = 2^-24, half a step of FP32):
  * norm and gate: FP64, rounded once to FP32, so the rows, the codes and the scales
    equal the definition's, up to values within 2^-50 of a rounding border, which
    seeded inputs do not hold;
  * rotary positions: the same, and the cache's bytes and words equal;
  * attention, componentwise, of W = sum_t p_t |v_t| over the softmax's weights p:
    a score is a sum of 2D products of FP16 pieces (22 of q's 24 bits, exact codes), scaled
    by two rounded factors, so it is off by at most (2D + 4 + 4) u of S = scale sum |q||k|
    (the pieces' 2^-23 is 2 u of it) plus, in powers of two, 3 roundings of a number of at
    most |score| log2(e) + 64 (the value's exponent; a running maximum of the same size);
    exp2 adds 2^-22.  With e the sum of these, numerator and denominator are each off by e
    and by one rounding a key; the pieces of a weight add 2^-22, the division and the join of
    up to 64 ranges (two roundings each) 130 u: (2 e + (2 n + 130) u + 2^-22) W.  A weight times its
    value's step, p s, is held in FP16 pieces whose quantum is 2^-24 where the row's largest is at
    least 2^5, so each is off by up to 2^-30 of that in absolute terms: with codes of at most 15,
    15 n 2^-30 max(p s) more (which shows where values differ by more than 2^20 in size);
  * attention, in norm: roundings that are independent add up by squares; with
    some 10^2 of them between input and output, 2e-6 of the norm of the result; and the 3
    roundings of a score in powers of two with a value's exponent, A = |score| log2(e) + |e|, each half
    a step of a number of up to A, do not average where a row is one or two keys: ln(2) 3 u A.
    (Scores of 100 and more: their sum over the features, in 2D/16 steps of which each may cut off up
    to a whole step of FP32, 2 u, at half its size on average, adds 2D/16 = D/8 roundings.)
"""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
from oracle import layer as RL
from tests.parity import say, to_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def host(t):
    torch.cuda.synchronize()
    t = t.detach().cpu()
    return t.float().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.numpy()


def rounded(t):
    return lambda h: torch.from_numpy(h).to(TYPES[t]).float().numpy()


def acts(rng, M, K, t="f32"):
    X = rng.standard_normal((M, K)).astype(np.float32)
    X[:, rng.permutation(K)[:max(1, K // 100)]] *= 30
    return rounded(t)(X)


def dev(a, t="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[t]).cuda()


def same_rows(qx, sx, y, name=""):
    """Codes and scales are those of the FP32 rows y."""
    q, s = RL.quant(y)
    assert np.array_equal(host(sx), s.astype(np.float32)), name
    bad = np.argwhere(host(qx).astype(np.int64) != q)
    assert not len(bad), (name, len(bad), bad[:4].tolist())


# ---------------------------------------------------------------- rows

@pytest.mark.parametrize("M,H,t,wt,res", [
    (1, 64, "f32", "f32", False), (1, 4096, "f32", "bf16", True), (3, 2560, "bf16", "bf16", True),
    (5, 5120, "f16", "f32", True), (257, 5120, "f32", "f16", True), (300, 2624, "bf16", "f32", False),
    (259, 16448, "f32", "f32", True), (2, 32768, "f16", "f16", True), (256, 16384, "f32", "f32", True),
])
def test_norm(M, H, t, wt, res):
    rng = np.random.default_rng(M + H)
    X, W = acts(rng, M, H, t), rounded(wt)((rng.random(H) + 0.5).astype(np.float32))
    R = acts(rng, M, H, t) * 2 if res else None
    h, y = RL.norm(X, W, R, 1e-5, rounded(t))
    Y = torch.empty((M, H), device="cuda")
    got = aq.aq_norm_quant(dev(X, t), dev(W, wt), None if R is None else dev(R, t), eps=1e-5, Y=Y)
    assert np.array_equal(host(Y), y)
    same_rows(got[0], got[1], y)
    if res:
        assert got[2].dtype == TYPES[t] and np.array_equal(host(got[2]), h)
        # in place of either, without Y
        for k in (0, 1):
            a, b = dev(X, t), dev(R, t)
            q, s, o = aq.aq_norm_quant(a, dev(W, wt), b, eps=1e-5, h=(a, b)[k])
            assert o.data_ptr() == (a, b)[k].data_ptr() and np.array_equal(host(o), h)
            assert torch.equal(q, got[0]) and torch.equal(s, got[1])
            assert np.array_equal(host((b, a)[k]), (R, X)[k])


@pytest.mark.parametrize("M", [2, 256])
def test_rows_of_every_length(M):
    """Norm and gate at both sides of each number of values a thread holds (whole turns of 256, 512 or
    1024 threads of four)."""
    rng = np.random.default_rng(M)
    for n in (1024, 1088, 2048, 2112, 3008, 3136, 4096, 4160, 6144, 6208, 8192, 8256, 10240, 10304, 12288, 12352, 16384, 16448, 20480, 20544,
              24576, 24640, 32768):
        X, W = acts(rng, M, n, "f32"), (rng.random(n) + 0.5).astype(np.float32)
        same_rows(*aq.aq_norm_quant(dev(X), dev(W), eps=1e-6), RL.norm(X, W, None, 1e-6)[1], f"norm {n}")
        GU = (rng.standard_normal((M, 2 * n)) * 3).astype(np.float32)
        same_rows(*aq.aq_swiglu_quant(dev(GU)), RL.swiglu(GU), f"gate {n}")


def test_norm_rows_that_stand_out():
    """Zero rows, tiny and huge rows, rows that are not finite beside others."""
    rng = np.random.default_rng(3)
    X, W = acts(rng, 8, 256), np.ones(256, np.float32)
    X[1] = 0
    X[2] *= 1e-30
    X[3] *= 1e30
    ref = RL.norm(X, W)[1]
    same_rows(*aq.aq_norm_quant(dev(X), dev(W)), ref, "eps")
    clean = aq.aq_norm_quant(dev(X), dev(W))
    X[4, 7], X[5, 9] = np.nan, np.inf
    q, s = aq.aq_norm_quant(dev(X), dev(W))
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])
    assert not np.isfinite(host(s)[[4, 5]]).any()
    q, s = aq.aq_norm_quant(dev(X[:3]), dev(W), eps=0.0)   # 0 / 0
    assert np.isnan(host(s)[1]) and np.isfinite(host(s)[[0, 2]]).all()


@pytest.mark.parametrize("M,I", [(1, 64), (5, 14336), (7, 9728), (255, 704), (256, 9728), (300, 17408), (2, 32768)])
def test_swiglu(M, I):
    rng = np.random.default_rng(M * I)
    GU = (rng.standard_normal((M, 2 * I)) * 3).astype(np.float32)
    GU[0, :6] = [-800, 800, -100, 0, -0.0, 1e-30]
    y = RL.swiglu(GU)
    Y = torch.empty((M, I), device="cuda")
    same_rows(*aq.aq_swiglu_quant(dev(GU), Y=Y), y)
    assert np.array_equal(host(Y), y)
    wide = torch.full((M, 2 * I + 64), 7.0, device="cuda")   # the two members' columns of a wider projection
    wide[:, 32:32 + 2 * I] = dev(GU)
    q, s = aq.aq_swiglu_quant(wide[:, 32:32 + 2 * I])
    same_rows(q, s, y)


def test_swiglu_values_near_ties_and_equal_maxima():
    """Rows whose largest magnitude is reached many times or within a step of it, and
    quotients on a tie: whatever estimate decides first, the rule decides last."""
    rng = np.random.default_rng(11)
    M, I = 64, 512
    g = np.full((M, I), 20.0, np.float32)                      # silu(20) rounds next to 20
    u = (rng.integers(-127, 128, (M, I)) + 0.5 * rng.integers(0, 2, (M, I))).astype(np.float32)
    u[:, ::7] = 127
    u[:, 1::7] = np.nextafter(np.float32(127), np.float32(rng.choice([0, 200])))
    g[32:] = (rng.random((32, I)) * 1e-3 + 20).astype(np.float32)
    GU = np.concatenate([g, u], 1)
    same_rows(*aq.aq_swiglu_quant(dev(GU)), RL.swiglu(GU))
    GU[5, 3], GU[6, I + 4] = np.nan, np.inf
    q, s = aq.aq_swiglu_quant(dev(GU))
    assert not np.isfinite(host(s)[[5, 6]]).any()
    keep = [i for i in range(M) if i not in (5, 6)]
    same_rows(q[keep], s[keep], RL.swiglu(GU[keep]))


# ---------------------------------------------------------------- rotary positions and the cache

def freqs(pairs, theta=1e6):
    return (1 / theta ** (np.arange(pairs) / pairs)).astype(np.float32)


def cache_of(pages, P, heads, D, seed=0):
    """A cache of noise: whatever is not written must neither change nor matter."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (pages, 2, heads, P, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    words = torch.full((pages, 2, heads, P), 0x7FC00000, dtype=torch.int32, device="cuda")
    return aq.aq_kv4_cache_of(codes, words)


@pytest.mark.parametrize("M,Hq,heads,D,parts,inter,P", [
    (1, 32, 8, 128, (64,), False, 64), (3, 7, 1, 128, (16, 24, 24), False, 16), (5, 14, 2, 64, (32,), True, 32),
    (33, 3, 3, 64, (5, 7, 3, 1), False, 128), (130, 40, 8, 128, (1, 20, 9), True, 256), (2000, 5, 1, 64, (8, 12, 12), False, 16),
    (9, 0, 2, 128, (32,), False, 16), (17, 2, 1, 64, None, False, 64), (4, 1, 1, 128, (1,), False, 16),
])
def test_rope_and_append(M, Hq, heads, D, parts, inter, P):
    rng = np.random.default_rng(M * 31 + Hq)
    x = acts(rng, M, (Hq + 2 * heads) * D).reshape(M, -1, D)
    x[0, -1] = 0                                       # a value of zeros
    if M > 2:
        x[1, Hq] = np.abs(x[1, Hq]) + 1                 # a key of one sign (before it turns)
        x[2, -1] = -np.abs(x[2, -1]) * 1e20
    pages = -(-M // P) + 3
    slots = rng.permutation(pages * P)[:M].astype(np.int64)
    if M > 4:
        slots[3], slots[4] = -1, pages * P              # padding rows
    cache = cache_of(pages, P, heads, D)
    codes0, words0 = host(cache.codes).copy(), host(cache.words).copy()
    if parts is None:
        r = rope = pos = None
        turned = x[:, :Hq + heads].astype(np.float32)
    else:
        f = freqs(sum(parts))
        pos = rng.integers(-5, 1 << 20, (len(parts), M)).astype(np.int32)
        rope = aq.aq_rope_axes(dev(f), parts, D, inter)
        turned = RL.rope(x[:, :Hq + heads], pos, f, parts, inter)
        pos = torch.from_numpy(pos).cuda()
    X = dev(x.reshape(M, -1))
    q = aq.aq_rope_kv4(X, rope, pos, cache, to_dev(slots))
    assert np.array_equal(host(q), turned[:, :Hq])
    assert np.array_equal(host(X), x.reshape(M, -1))
    kv = np.stack([turned[:, Hq:], x[:, Hq + heads:]], 1)        # [M, 2, heads, D]
    c, w = RL.hold(kv)
    codes1, words1 = codes0.copy(), words0.view(np.uint32).copy()
    for m in np.flatnonzero((slots >= 0) & (slots < pages * P)):
        codes1[slots[m] // P, :, :, slots[m] % P] = RL.packed(c[m])
        words1[slots[m] // P, :, :, slots[m] % P] = w[m]
    assert np.array_equal(host(cache.words).view(np.uint32), words1)
    assert np.array_equal(host(cache.codes), codes1)
    # read back
    K, V = aq.aq_kv4_read(cache, to_dev(slots))
    want = RL.values(RL.packed(c), w)
    want[(slots < 0) | (slots >= pages * P)] = 0
    got = np.stack([host(K), host(V)], 1)
    assert np.array_equal(got, want.astype(np.float32), equal_nan=True)
    # (a vector whose scale would pass 2^64, as the one times 1e20 may, is held as NaN)
    # the rows' distance from what is held: half a step, and where the range is cut at 15 steps up to another half
    step = (w & ~np.uint32(15)).view(np.float32)[..., None]
    inside = ((slots >= 0) & (slots < pages * P))[:, None, None] & np.isfinite(want).all(-1)
    assert (np.abs(want - kv)[inside] <= 1.0001 * step[inside]).all()
    # in place, in a wider row
    if Hq:
        wide = torch.full((M, X.shape[1] + 8), 3.0, device="cuda")
        wide[:, 4:-4] = X
        view = wide[:, 4:-4]
        again = cache_of(pages, P, heads, D)
        out = view.unflatten(1, (-1, D))[:, :Hq]
        got = aq.aq_rope_kv4(view, rope, pos, again, to_dev(slots), out=out)
        assert got.data_ptr() == view.data_ptr() and torch.equal(got, q)
        assert torch.equal(view[:, Hq * D:], X[:, Hq * D:]) and (wide[:, :4] == 3).all() and (wide[:, -4:] == 3).all()
        assert torch.equal(again.codes, cache.codes) and torch.equal(again.words, cache.words)


def test_append_vectors_that_are_not_finite_and_ties():
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 3, 128)).astype(np.float32)
    x[1, 1, 5], x[2, 2, 7], x[3, 1, 0] = np.nan, np.inf, -np.inf
    x[4, 1] = np.tile([-7.5, 7.5, 0.5, -0.5, 1.5, 2.5, -1.5, 0], 16)      # s a little over 1
    x[5, 1] = np.tile([0, 15, 0.5, 1.5, 2.5, 3.5, 14.5, 7.5], 16)
    x[5, 2] = 1e-20
    cache = aq.aq_kv4_cache(1, 16, 1, 128)
    aq.aq_rope_kv4(dev(x.reshape(6, -1)), None, None, cache, torch.arange(6, device="cuda"))
    c, w = RL.hold(x[:, 1:])
    got = host(cache.words).view(np.uint32)[0, :, 0, :6].T
    assert np.array_equal(got, w) and (got == 0x7FC00000).sum() == 3
    assert np.array_equal(host(cache.codes)[0, :, 0, :6].transpose(1, 0, 2), RL.packed(c))


# ---------------------------------------------------------------- attention

def pages_for(rng, lens, P, extra=2):
    need = [-(-n // P) for n in lens]
    total = sum(need) + 3
    order, table, at = rng.permutation(total).astype(np.int32), np.full((len(lens), max(need + [1]) + extra), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def filled(rng, lens, P, heads, D, spread=1.0):
    """Pages whose held tokens are random codes and words; all other words NaN."""
    table, total = pages_for(rng, lens, P)
    codes = rng.integers(0, 256, (total, 2, heads, P, D // 2)).astype(np.uint8)
    words = np.full((total, 2, heads, P), 0x7FC00000, np.uint32)
    for b, n in enumerate(lens):
        at = np.arange(n)
        s = (0.3 * np.exp(spread * rng.standard_normal((n, 2, heads)))).astype(np.float32)
        s[:, 0] = 0.2 * (rng.random((n, heads)) + 0.5)
        words[table[b, at // P], :, :, at % P] = (s.view(np.uint32) & ~np.uint32(15)) | rng.integers(0, 16, s.shape).astype(np.uint32)
    return table, codes, words


def as_cache(codes, words):
    return aq.aq_kv4_cache_of(torch.from_numpy(codes).cuda(), torch.from_numpy(words.view(np.int32)).cuda())


def check_attn(q, codes, words, table, lens, cu=None, scale=None, name="", got=None, roundings=3):
    M, Hq, D = q.shape
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    if got is None:
        out = torch.full((M, Hq * D), 123.0, device="cuda")
        got = aq.aq_attn_kv4(dev(q), as_cache(codes, words), i32(table), i32(lens), None if cu is None else i32(cu), scale=scale,
                             out=out)
    got = host(got).reshape(M, Hq, D).astype(np.float64)
    sums = {}
    ref = RL.attention(q, codes, words, table, lens, cu, scale, sums).reshape(M, Hq, D)
    owned = ~np.isnan(ref).all((1, 2)) if cu is not None else np.ones(M, bool)
    if cu is not None:
        owned = np.zeros(M, bool)
        for b in range(len(lens)):
            owned[cu[b]:cu[b + 1]] = True
    assert (got[~owned] == 123.0).all(), name
    worst = most = 0.0
    for m in np.flatnonzero(owned):
        for j in range(Hq):
            if (m, j) not in sums:
                assert (got[m, j] == 0).all(), (name, m, j)
                continue
            W, S, n, top, A = sums[m, j]
            most = max(most, A) if np.isfinite(A) else most
            if np.isnan(ref[m, j]).any():
                assert np.isnan(got[m, j]).all(), (name, m, j)
                continue
            e = np.log(2) * 3 * U * (np.max(S) * 1.4427 + 64) + (2 * D + 8) * U * np.max(S) + 2.0 ** -22
            tol = (2 * e + (2 * n + 130) * U + 2.0 ** -22) * W + 15 * n * 2.0 ** -30 * top + 1e-30
            err = np.abs(got[m, j] - ref[m, j])
            worst = max(worst, float((err / tol).max()))
            assert (err <= tol).all(), (name, m, j, float(err.max()), float((err / tol).max()))
    fine = owned[:, None, None] & np.isfinite(ref)
    rel = np.linalg.norm((got - ref)[fine]) / max(np.linalg.norm(ref[fine]), 1e-300)
    say(f"  attention {name}: {rel:.2e} in norm, worst {worst:.3f} of the componentwise bound")
    assert rel <= 2e-6 + np.log(2) * roundings * U * most, (name, rel)
    return got


CASES = [
    # lens, new tokens (None: one each), Hq, heads, D, P
    ([1], None, 1, 1, 64, 16),
    ([17], None, 4, 1, 128, 16),
    ([700, 1, 0, 129, 128], None, 32, 8, 128, 64),
    ([64, 65, 63, 300], None, 14, 2, 64, 32),
    ([2000, 31], None, 17, 1, 128, 128),
    ([5000], None, 10, 2, 128, 256),
    ([260, 900], None, 66, 2, 64, 16),
    # short chunks
    ([5, 40, 9], [5, 3, 0], 8, 2, 128, 16),
    ([300, 20, 1], [4, 1, 1], 6, 2, 64, 64),
    # prompts
    ([33], [33], 4, 1, 128, 16),
    ([150, 70, 200], [150, 1, 77], 4, 2, 128, 32),
    ([130, 300], [130, 260], 7, 1, 64, 64),
    ([600], [300], 3, 3, 128, 64),
    ([400, 0, 64, 8], [129, 0, 64, 8], 16, 2, 64, 128),
    ([70], [70], 32, 8, 128, 16),
    ([150, 70, 200], [150, 1, 77], 10, 2, 128, 32),
    ([600], [300], 7, 7, 128, 64),
    # fewer cached tokens than queries: rows in front of the first key
    ([10, 3], [40, 50], 24, 1, 128, 16),
    ([0, 300], [60, 150], 10, 2, 64, 16),
    ([10, 3], [40, 50], 4, 1, 128, 16),
    ([0, 2], [3, 2], 2, 1, 64, 16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_attention(case):
    lens, new, Hq, heads, D, P = case
    rng = np.random.default_rng(sum(lens) + Hq)
    table, codes, words = filled(rng, lens, P, heads, D)
    cu = None if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    M = len(lens) if new is None else int(cu[-1]) + 3        # three rows behind the last sequence
    q = rng.standard_normal((M, Hq, D)).astype(np.float32)
    check_attn(q, codes, words, table, lens, cu, name=str(case))
