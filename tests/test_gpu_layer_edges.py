"""Where a decoder layer's steps can go wrong beside test_gpu_layer.py (whose
tolerances these tests share): values that are not finite and values of
extreme size, pages and lengths out of range, many and empty sequences, offsets past
32 bits, strides, graphs and streams, and a prompt taken whole, in chunks and token by
token."""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
from oracle import layer as RL
from tests.parity import to_dev
from tests.test_gpu_layer import acts, as_cache, cache_of, check_attn, dev, filled, freqs, host, same_rows

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def call(q, codes, words, table, lens, cu=None, **k):
    return aq.aq_attn_kv4(q if torch.is_tensor(q) else dev(q), as_cache(codes, words), i32(table), i32(lens), None if cu is None else i32(cu), **k)


# rows (single tokens, chunks) and tiles (prompts) of the attention kernels
SHAPES = [dict(lens=[300, 77], new=None, Hq=8, heads=2, D=128, P=16), dict(lens=[300, 77], new=[3, 2], Hq=6, heads=2, D=64, P=32),
          dict(lens=[300, 77], new=[150, 77], Hq=4, heads=2, D=128, P=64), dict(lens=[400, 90], new=[400, 60], Hq=2, heads=1, D=64, P=16),
          # (more than 2048 rows of query heads in all: tiles of 128 rows)
          dict(lens=[300, 77], new=[150, 77], Hq=10, heads=2, D=128, P=64), dict(lens=[400, 90], new=[400, 60], Hq=5, heads=1, D=64, P=16)]


def made(s, seed=0, spread=1.0):
    rng = np.random.default_rng(seed)
    table, codes, words = filled(rng, s["lens"], s["P"], s["heads"], s["D"], spread)
    cu = None if s["new"] is None else np.concatenate([[0], np.cumsum(s["new"])]).astype(np.int32)
    M = len(s["lens"]) if cu is None else int(cu[-1])
    q = rng.standard_normal((M, s["Hq"], s["D"])).astype(np.float32)
    return rng, q, codes, words, table, np.array(s["lens"]), cu


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s['new']}-{s['D']}")
@pytest.mark.parametrize("what", ["query", "key", "value", "both"])
def test_not_finite(s, what):
    """A query, key or value that is not finite makes NaN of the rows that see it and
    leaves every other row as it was, bit for bit."""
    rng, q, codes, words, table, lens, cu = made(s)
    heads, G, P = s["heads"], s["Hq"] // s["heads"], s["P"]
    clean = host(call(q, codes, words, table, lens, cu)).reshape(q.shape)
    bad = np.zeros(q.shape[:2], bool)
    if what == "query":
        q[0, 1, 3], q[-1, 0, 0], q[-1, s["Hq"] - 1, 1] = np.nan, np.inf, -np.inf
        bad[0, 1] = bad[-1, 0] = bad[-1, -1] = True
    else:
        t = 220 if s["new"] else 299                    # among the first sequence's tokens
        page = table[0, t // P]
        for kv in ([0], [1], [0, 1])[["key", "value", "both"].index(what)]:
            words[page, kv, heads - 1, t % P] = 0x7FC00000
        n = 1 if cu is None else s["new"][0]
        for i in range(n):
            if t <= lens[0] - n + i:
                bad[i, (heads - 1) * G:] = True
        assert bad.any()
    got = host(call(q, codes, words, table, lens, cu)).reshape(q.shape)
    assert np.isnan(got[bad]).all()
    assert np.array_equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s['new']}-{s['D']}")
def test_extreme_sizes(s):
    """Scales of values from nothing to 1e18 side by side, and beyond 2^64, which are NaN; rows of q
    far larger and smaller than their neighbours, whose results they leave as they were."""
    rng, q, codes, words, table, lens, cu = made(s, 1, spread=6.0)
    P = s["P"]
    for t, sc in ((2, 1e18), (5, 1e-12), (11, 0.0), (12, 1e-19), (33, 1e17), (60, 1e-30)):
        w = np.float32(sc).view(np.uint32) & ~np.uint32(15) | np.uint32(9)
        for b in range(2):
            words[table[b, t // P], 1, :, t % P] = w
    check_attn(q, codes, words, table, lens, cu, name="far apart")
    words[table[0, 1 // P], 0, 0, 1 % P] = np.float32(0).view(np.uint32)   # a key of nothing
    check_attn(q, codes, words, table, lens, cu, name="a key of nothing")
    beyond = words.copy()
    for t, sc in ((3, 1e-12), (10, 0.0), (40, 1e30), (41, 1e-30), (70, 3e37)):
        w = np.float32(sc).view(np.uint32) & ~np.uint32(15) | np.uint32(5)
        for b in range(2):
            beyond[table[b, t // P], 1, :, t % P] = w
    check_attn(q, codes, beyond, table, lens, cu, name="scales past 2^64")
    beyond = words.copy()
    beyond[table[0, 20 // P], 0, 0, 20 % P] = np.float32(-0.5).view(np.uint32)
    check_attn(q, codes, beyond, table, lens, cu, name="a negative scale")
    clean = host(call(q, codes, words, table, lens, cu)).reshape(q.shape)
    q2 = q.copy()
    q2[0, 0] *= 1e-30
    q2[-1, -1] *= 1e4
    q2[-1, 0] *= np.float32(1e-3)
    got = check_attn(q2, codes, words, table, lens, cu, name="rows")
    same = np.ones(q.shape[:2], bool)
    same[0, 0] = same[-1, -1] = same[-1, 0] = False
    assert np.array_equal(got[same].astype(np.float32), clean[same])
    q3 = q.copy()
    q3[0, 0], q3[-1, -1] = 1e30, -1e36                     # scores past every exponential
    got = host(call(q3, codes, words, table, lens, cu)).reshape(q.shape)
    assert np.array_equal(got[same], clean[same])
    z = np.zeros_like(q)                                   # all scores equal: the mean of the values
    check_attn(z, codes, words, table, lens, cu, name="zeros")
    check_attn(q, codes, words, table, lens, cu, scale=0.0, name="no scale")
    check_attn(q, codes, words, table, lens, cu, scale=1.0, name="peaked", roundings=3 + s["D"] // 8)


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s['new']}-{s['D']}")
def test_pages_and_lengths_out_of_range(s):
    rng, q, codes, words, table, lens, cu = made(s, 2)
    for at, page in ((0, -1), (1, codes.shape[0]), (2, 1 << 30), (4, -(1 << 31))):
        if at < -(-lens[0] // s["P"]):
            table[0, at] = page
    check_attn(q, codes, words, table, lens, cu, name="pages")
    table[1] = -7
    check_attn(q, codes, words, table, lens, cu, name="no page at all")
    rng, q, codes, words, table, lens, cu = made(s, 3)
    most = table.shape[1] * s["P"]
    for b, n in ((0, -5), (1, 1 << 30)):
        changed = lens.copy()
        changed[b] = n
        got = host(call(q, codes, words, table, changed, cu)).reshape(q.shape)
        changed[b] = min(max(n, 0), most)
        check_attn(q, codes, words, table, changed, cu, name=f"length {n}", got=torch.from_numpy(got).cuda())


@pytest.mark.parametrize("s", [SHAPES[2], SHAPES[4]], ids=["rows", "tiles"])
def test_offsets_that_do_not_increase(s):
    """Row offsets that the call does not allow change nothing but rows: every
    address stays inside its tensor."""
    rng, q, codes, words, table, lens, cu = made(s, 4)
    M = q.shape[0]
    guard = torch.full((3 * M, s["Hq"] * s["D"]), 5.0, device="cuda")
    for bad in ([0, M + 9, M], [-4, 20, 10], [30, 20, 1 << 30], [0, 0, 0], [M, M, M]):
        call(q, codes, words, table, lens, bad, out=guard[M:2 * M])
        torch.cuda.synchronize()
        assert (guard[:M] == 5).all() and (guard[2 * M:] == 5).all()
    rows = torch.full((M, s["Hq"] * s["D"]), 5.0, device="cuda")
    call(q, codes, words, table, lens, [0, 0, 0], out=rows)
    assert (rows == 5).all()


@pytest.mark.parametrize("B,Hq,heads,D,P,longest,width", [
    (100, 3, 1, 64, 16, 700, 0), (300, 2, 1, 64, 16, 900, 0), (257, 5, 1, 128, 32, 60, 4000), (64, 16, 16, 64, 16, 200, 0),
    (70, 8, 1, 128, 256, 3000, 0), (2, 64, 1, 128, 64, 9000, 0), (3, 12, 4, 128, 16, 30000, 0),
])
def test_many_single_tokens(B, Hq, heads, D, P, longest, width):
    """Batches whose workgroups find their place by search (up to 128 sequences, where contexts may be cut) and by number."""
    rng = np.random.default_rng(B)
    lens = (longest ** rng.random(B)).astype(int)
    lens[rng.integers(0, B, max(1, B // 7))] = 0
    lens[B // 2] = longest
    table, codes, words = filled(rng, lens, P, heads, D)
    if width:
        table = np.concatenate([table, np.full((B, width), -1, np.int32)], 1)   # room for far more keys
    check_attn(rng.standard_normal((B, Hq, D)).astype(np.float32), codes, words, table, lens, name=f"B {B}")


@pytest.mark.parametrize("new,old,Hq,heads,D,P", [
    ([0] * 70 + [1, 0, 5] + [0] * 80 + [2], 40, 4, 2, 64, 16), ([1] * 130 + [3], 300, 5, 1, 128, 32), ([200] + [0] * 64 + [90], 100, 2, 1, 64, 16),
    ([40] * 70, 260, 16, 16, 64, 16), ([200] + [0] * 64 + [90], 100, 8, 1, 64, 16), ([1, 700], 10, 4, 1, 128, 64),
    ([1, 700], 10, 1, 1, 128, 64), ([31, 33, 129, 1, 1, 1], 0, 9, 1, 64, 128),
])
def test_many_ragged_sequences(new, old, Hq, heads, D, P):
    rng = np.random.default_rng(len(new))
    lens = np.array([n + (int(rng.integers(0, old + 1)) if n else 0) for n in new])
    table, codes, words = filled(rng, lens, P, heads, D)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    check_attn(rng.standard_normal((int(cu[-1]) + 2, Hq, D)).astype(np.float32), codes, words, table, lens, cu, name=f"{len(new)} sequences")


@pytest.mark.parametrize("B,chunk,old,Hq,heads,D,P", [
    (257, 1, 300, 4, 2, 64, 16), (1000, 3, 5, 2, 1, 64, 16), (4097, 1, 2, 1, 1, 64, 16), (300, 1, 6000, 3, 1, 128, 64), (300, 200, 40, 2, 1, 64, 32),
])
def test_many_packed_sequences(B, chunk, old, Hq, heads, D, P):
    """Packed sequences beyond the 128 that a workgroup sums itself: indexed first, for few rows each and
    for prompts; sequences without rows or keys among them, also the first and the last."""
    rng = np.random.default_rng(B + chunk)
    new = rng.integers(0, chunk + 1, B)
    lens = new + (rng.integers(0, old + 1, B) if old < 1000 else (old ** rng.random(B)).astype(int))
    new[[0, B - 1]] = 0
    lens[B // 3] = 0
    new[B // 2], lens[B // 2] = chunk, chunk + old
    lens = np.maximum(lens, new * (np.arange(B) != B // 3))
    table, codes, words = filled(rng, lens, P, heads, D)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]) + 2, Hq, D)).astype(np.float32)
    check_attn(q, codes, words, table, lens, cu, name=f"{B} sequences")
    cache, d = aq.aq_kv4_cache_of(to_dev(codes), to_dev(words.view(np.int32))), dev(q)
    args = (d, cache, i32(table), i32(lens), i32(cu))
    want = aq.aq_attn_kv4(*args, out=torch.full((q.shape[0], Hq * D), 5.0, device="cuda"))
    assert (want[int(cu[-1]):] == 5).all()
    guard = torch.full((3 * q.shape[0], Hq * D), 5.0, device="cuda")
    for bad in (cu[::-1].copy(), cu * 4096, np.where(np.arange(B + 1) % 2, cu[-1], 0)):
        aq.aq_attn_kv4(*args[:4], i32(bad), out=guard[q.shape[0]:2 * q.shape[0]])
        torch.cuda.synchronize()
        assert (guard[:q.shape[0]] == 5).all() and (guard[2 * q.shape[0]:] == 5).all()
    st = torch.cuda.Stream()
    out = torch.full((q.shape[0], Hq * D), 5.0, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            aq.aq_attn_kv4(*args, out=out)
        for _ in range(3):
            out.fill_(5.0)
            g.replay()
            st.synchronize()
            assert torch.equal(out, want)


@pytest.mark.parametrize("B,new,old,Hq,heads,D,P", [
    (20, [200], 300, 8, 2, 128, 16), (16, [130, 5, 90], 700, 14, 2, 64, 32), (40, [17, 16, 15, 300, 4], 200, 8, 8, 128, 64), (18, [400], 60, 17, 1, 64, 16),
    (17, [120], 90, 40, 1, 64, 64), (300, [3000, 8, 9], 40, 4, 1, 64, 16), (25, [500], 6000, 4, 1, 64, 128), (16, [300] * 16, 30, 4, 2, 64, 16),
])
def test_single_tokens_beside_prompts(B, new, old, Hq, heads, D, P):
    """Batches of single tokens with some prompts among them: the sequences of few rows are a launch of
    their own, without the others' rows, and each row is one launch's alone."""
    rng = np.random.default_rng(B + len(new))
    n = np.ones(B, int)
    n[rng.permutation(B)[:len(new)]] = new
    n[rng.integers(0, B)] = 0
    lens = n + (old ** rng.random(B)).astype(int)
    lens[B // 2] = n[B // 2] + old
    table, codes, words = filled(rng, lens, P, heads, D)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]) + 1, Hq, D)).astype(np.float32)
    check_attn(q, codes, words, table, lens, cu, name=f"{B} sequences, {new[:4]}")
    # captured, and again
    args = (dev(q), aq.aq_kv4_cache_of(to_dev(codes), to_dev(words.view(np.int32))), i32(table), i32(lens), i32(cu))
    out = torch.full((q.shape[0], Hq * D), 5.0, device="cuda")
    want = aq.aq_attn_kv4(*args, out=out).clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            aq.aq_attn_kv4(*args, out=out)
        for _ in range(3):
            out.fill_(5.0)
            g.replay()
            st.synchronize()
            assert torch.equal(out, want)


def test_cache_past_32_bits():
    """A cache of 4.4 GB: pages behind 2^32 bytes of codes, appended to, read and attended."""
    P, heads, D, Hq = 256, 8, 128, 8
    pages = (1 << 32) // (2 * heads * P * D // 2) + 600
    codes = torch.empty((pages, 2, heads, P, D // 2), dtype=torch.uint8, device="cuda")
    words = torch.empty((pages, 2, heads, P), dtype=torch.int32, device="cuda")
    cache = aq.aq_kv4_cache_of(codes, words)
    rng = np.random.default_rng(12)
    n = 600
    table = np.array([[pages - 1, 3, pages - 577]], np.int32)
    slots = table[0, np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
    x = acts(rng, n, (Hq + 2 * heads) * D)
    q = aq.aq_rope_kv4(dev(x), None, None, cache, to_dev(slots))
    kv = x.reshape(n, -1, D)[:, Hq:].reshape(n, 2, heads, D)
    c, w = RL.hold(kv)
    K, V = aq.aq_kv4_read(cache, to_dev(slots))
    assert np.array_equal(np.stack([host(K), host(V)], 1), RL.values(RL.packed(c), w).astype(np.float32))
    small_c, small_w = np.zeros((3, 2, heads, P, D // 2), np.uint8), np.zeros((3, 2, heads, P), np.uint32)
    for t in range(n):
        small_c[t // P, :, :, t % P], small_w[t // P, :, :, t % P] = RL.packed(c[t]), w[t]
    small_t = np.array([[0, 1, 2]], np.int32)
    for rows, cu in ((slice(n - 1, n), None), (slice(0, n), [0, n])):
        got = aq.aq_attn_kv4(q[rows].contiguous(), cache, i32(table), i32([n]), None if cu is None else i32(cu))
        check_attn(host(q[rows]), small_c, small_w, small_t, np.array([n]), None if cu is None else np.array(cu), name="4.4 GB", got=got)


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s['new']}-{s['D']}")
def test_queries_in_wider_rows_and_given_buffers(s):
    rng, q, codes, words, table, lens, cu = made(s, 5)
    want = call(q, codes, words, table, lens, cu)
    wide = torch.full((q.shape[0], s["Hq"] * s["D"] + 40), float("nan"), device="cuda")
    wide[:, 20:20 + s["Hq"] * s["D"]] = dev(q).flatten(1)
    view = wide[:, 20:20 + s["Hq"] * s["D"]].unflatten(1, (s["Hq"], s["D"]))
    out, ws = torch.empty_like(want), torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    got = call(view, codes, words, table, lens, cu, out=out, ws=ws)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
    assert torch.equal(call(view, codes, words, table, lens, cu, out=out, ws=ws), want)   # what a call leaves there does not matter
    with pytest.raises(ValueError):
        call(view.transpose(0, 1), codes, words, table, lens, cu)
    with pytest.raises(ValueError):
        call(dev(q).half(), codes, words, table, lens, cu)


def test_prompt_whole_in_chunks_and_by_tokens():
    """The run of the steps together on one sequence: rotary positions, append and attention of a
    prompt in one call, in chunks, and token by token: the same cache, bit for bit, and outputs that
    differ by the order of sums alone."""
    rng = np.random.default_rng(21)
    n, Hq, heads, D, P = 310, 8, 2, 128, 16
    x = dev(acts(rng, n, (Hq + 2 * heads) * D))
    f = to_dev(freqs(64, 1e4))
    rope = aq.aq_rope_axes(f, (64,), D)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    pages = -(-n // P)
    table = torch.randperm(pages, device="cuda").int()[None]
    slots = table[0, (pos // P).long()].long() * P + pos % P

    def run(cuts):
        cache, outs = cache_of(pages, P, heads, D), []
        for a, b in zip(cuts, cuts[1:]):
            q = aq.aq_rope_kv4(x[a:b], rope, pos[a:b].contiguous(), cache, slots[a:b].contiguous())
            outs.append(aq.aq_attn_kv4(q, cache, table, i32([b]), None if b - a == 1 else i32([0, b - a])))
        return cache, torch.cat(outs)

    whole, o = run([0, n])
    ref = host(o).astype(np.float64)
    for cuts in ([0, 1, 2, 7, 16, 140, 141, 300, n], list(range(0, n + 1))):
        cache, got = run(cuts)
        seen = slots.cpu().numpy()
        assert np.array_equal(host(cache.codes)[seen // P, :, :, seen % P], host(whole.codes)[seen // P, :, :, seen % P])
        assert np.array_equal(host(cache.words)[seen // P, :, :, seen % P], host(whole.words)[seen // P, :, :, seen % P])
        err = np.linalg.norm(host(got) - ref) / np.linalg.norm(ref)
        assert err <= 4e-6, err                      # two errors in norm of 2e-6
    qq = RL.rope(host(x).reshape(n, -1, D)[:, :Hq], [np.arange(n)], host(f), (64,))
    check_attn(qq, host(whole.codes), host(whole.words).view(np.uint32), host(table), np.array([n]), np.array([0, n]), name="whole", got=o)


def test_graphs_and_streams():
    """Two captured calls replayed side by side with eager work between, on other streams than
    the current one; every replay equals the eager result."""
    cases = [made(s, 6 + i) for i, s in enumerate(SHAPES)]
    rng = np.random.default_rng(30)
    x, w = dev(acts(rng, 70, 2560)), dev(np.ones(2560, np.float32))
    gu = dev(rng.standard_normal((9, 2 * 704)).astype(np.float32))
    qkv = dev(acts(rng, 33, 12 * 128))
    rope = aq.aq_rope_axes(to_dev(freqs(64)), (20, 44), 128)
    pos, slots = torch.arange(66, device="cuda").int().view(2, 33), torch.randperm(64, device="cuda")[:33]
    cache = cache_of(4, 16, 2, 128)
    handles = [(dev(c[1]), as_cache(c[2], c[3]), i32(c[4]), i32(c[5]), None if c[6] is None else i32(c[6])) for c in cases]

    def work():
        o = [aq.aq_attn_kv4(q, k, t, n, cu) for q, k, t, n, cu in handles]
        o += list(aq.aq_norm_quant(x, w, residual=x)) + list(aq.aq_swiglu_quant(gu))
        o.append(aq.aq_rope_kv4(qkv, rope, pos, cache, slots))
        return o + list(aq.aq_kv4_read(cache, slots))

    eager = [t.clone() for t in work()]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            work()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs = work()
        graphs.append((st, g, outs))
    for _ in range(4):
        for st, g, outs in graphs:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for st, g, outs in graphs:
            with torch.cuda.stream(st):
                g.replay()
        again = work()                                # eager, on the current stream, meanwhile
        torch.cuda.synchronize()
        for outs in [again] + [g[2] for g in graphs]:
            for a, b in zip(outs, eager):
                assert torch.equal(a, b)
    other = torch.cuda.Stream()
    q, k, t, n, cu = handles[0]
    other.wait_stream(torch.cuda.current_stream())
    got = aq.aq_attn_kv4(q, k, t, n, cu, stream=other)
    other.synchronize()
    assert torch.equal(got, eager[0])


def test_no_rows():
    assert aq.aq_norm_quant(torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda"))[0].shape == (0, 64)
    assert aq.aq_swiglu_quant(torch.empty((0, 128), device="cuda"))[1].shape == (0,)
    cache = cache_of(2, 16, 1, 64)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert aq.aq_rope_kv4(torch.empty((0, 192), device="cuda"), None, None, cache, none).shape == (0, 1, 64)
    assert aq.aq_kv4_read(cache, none)[0].shape == (0, 1, 64)
    o = aq.aq_attn_kv4(torch.empty((0, 1, 64), device="cuda"), cache, i32([[0]]), i32([5]), i32([0, 0]))
    assert o.shape == (0, 64)


def test_refused_by_the_binding():
    d = torch.empty
    X, W = d((2, 64), device="cuda"), d(64, device="cuda")
    cache = cache_of(2, 16, 1, 64)
    qkv, slots = d((2, 192), device="cuda"), torch.arange(2, device="cuda")
    rope = aq.aq_rope_axes(d(32, device="cuda"), (32,), 64)
    pos, q = torch.zeros((1, 2), dtype=torch.int32, device="cuda"), d((2, 1, 64), device="cuda")
    table, lens = i32([[0], [1]]), i32([3, 4])
    for f in (lambda: aq.aq_norm_quant(X.double(), W), lambda: aq.aq_norm_quant(X, W.cpu()), lambda: aq.aq_norm_quant(X, W[:32]),
              lambda: aq.aq_norm_quant(X, W, residual=X.half()), lambda: aq.aq_norm_quant(X, W, h=X), lambda: aq.aq_norm_quant(X.t(), W),
              lambda: aq.aq_swiglu_quant(X.t()), lambda: aq.aq_swiglu_quant(X.half()), lambda: aq.aq_swiglu_quant(X[:, :63]),
              lambda: aq.aq_rope_kv4(qkv, rope, pos.long(), cache, slots), lambda: aq.aq_rope_kv4(qkv, rope, pos, cache, slots.int()),
              lambda: aq.aq_rope_kv4(qkv, rope, pos.expand(2, 2).contiguous(), cache, slots), lambda: aq.aq_rope_kv4(qkv[:, :100], rope, pos, cache, slots),
              lambda: aq.aq_rope_kv4(qkv, rope, pos, cache, slots, out=d((2, 2, 64), device="cuda")), lambda: aq.aq_kv4_read(cache, slots.int()),
              lambda: aq.aq_kv4_cache(2, 16, 1, 64).__class__(cache.codes, cache.words[:1]), lambda: aq.aq_attn_kv4(q, cache, table.long(), lens),
              lambda: aq.aq_attn_kv4(q, cache, table, lens[:1]), lambda: aq.aq_attn_kv4(q, cache, table, lens, i32([0, 2])),
              lambda: aq.aq_attn_kv4(q[..., :32], cache, table, lens), lambda: aq.aq_attn_kv4(q.cpu(), cache, table, lens)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: aq.aq_norm_quant(X[:, :40].contiguous(), W[:40]), lambda: aq.aq_attn_kv4(q, cache, table, lens, scale=-1.0),
              lambda: aq.aq_attn_kv4(q, cache, table, lens, scale=float("nan")), lambda: aq.aq_attn_kv4(q[:1], cache, table, lens),
              lambda: aq.aq_rope_kv4(qkv, rope, pos, aq.aq_kv4_cache(2, 24, 1, 64), slots)):
        with pytest.raises(aq.AqError):
            f()
