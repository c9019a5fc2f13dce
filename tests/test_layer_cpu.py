"""A decoder layer's steps between its projections without a GPU: the oracle
pinned to hand-worked cases, the library's refusals (every one before a launch),
and its host file under AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import dataclasses
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from mixed_precision_int_amd import binding as B
from oracle import layer as RL

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # 16-byte-aligned fake device address; never dereferenced
FAR = 1 << 44


# ---------------------------------------------------------------- oracle

def test_norm_by_hand():
    h, y = RL.norm([[1, -1, 4, 2]], [1, 2, 1, 0.5], [[2, -2, -4, 0]], eps=2.5)
    assert h.tolist() == [[3, -3, 0, 2]]
    # mean of squares 22 / 4 = 5.5, 1 / sqrt(8)
    assert np.allclose(y, np.array([[3, -6, 0, 1]]) / np.sqrt(8), rtol=1e-7)
    q, s = RL.quant(y)
    # half of the largest is 63.5 steps, a tie but for the step's own rounding
    assert q[0, 0] in (63, 64) and q[0, 1:].tolist() == [-127, 0, 21] and np.isclose(s[0], 6 / np.sqrt(8) / 127)


def test_swiglu_by_hand():
    y = RL.swiglu([[0, np.log(3), -np.log(3), 5, 4, 8]])
    assert np.allclose(y, [[0, np.log(3) * 0.75 * 4, -np.log(3) * 0.25 * 8]], rtol=1e-7)


def test_rope_by_hand():
    x = np.array([[[1, 2, 3, 4, 5, 6]]], dtype=np.float32)
    f = [np.pi / 2, np.pi / 6]
    # axis 0 turns pair 0 by 90 degrees, axis 1 pair 1 by 180; the last two features stay
    want = [-3, -2, 1, -4, 5, 6]
    assert np.allclose(RL.rope(x, [[1], [6]], f, (1, 1)), [[want]], atol=1e-6)
    assert np.allclose(RL.rope(x, [[1], [6]], f, (1, 1), True), [[[-2, 1, -3, -4, 5, 6]]], atol=1e-6)
    # positions that FP32 angles would lose
    far = RL.rope(x, [[(1 << 24) + 1]], np.float32([1.0]), (1,))
    a = np.longdouble((1 << 24) + 1)
    assert np.allclose(far[0, 0, :2], [np.cos(a) * 1 - np.sin(a) * 2, np.cos(a) * 2 + np.sin(a) * 1], atol=1e-6)


def test_held_by_hand():
    x = np.zeros((4, 64), np.float32)
    x[0, :6] = [15, 0, 1.25, 7.5, -0.25, 0.5]          # lo -0.25, hi 15
    x[1, :3] = [30, 15, 3]                            # no negative: s = 2, z = 0
    x[2, :3] = [-7.5, -1, -0.25]                      # no positive: s = 0.5, z = 15
    c, w = RL.hold(x)
    s = (w & ~np.uint32(15)).view(np.float32)
    assert 0 <= s[0] - 15.25 / 15 < 2e-6 and w[0] & 15 == 0 and c[0, :6].tolist() == [15, 0, 1, 7, 0, 0]
    assert s[1] == 2 and w[1] & 15 == 0 and c[1, :3].tolist() == [15, 8, 2]       # 7.5 and 1.5 to even
    assert s[2] == 0.5 and w[2] & 15 == 15 and c[2, :4].tolist() == [0, 13, 15, 15]   # -0.5 to even
    assert 0 <= s[3] - 1e-12 < 2e-18 and (c[3] == 0).all()
    v = RL.values(RL.packed(c), w)
    assert np.abs(v[0] - x[0]).max() <= 0.52 * s[0] and v[1, :3].tolist() == [30, 16, 4] and v[2, :3].tolist() == [-7.5, -1, 0]
    assert RL.packed(np.arange(8)[None]).tolist() == [[0x10, 0x32, 0x54, 0x76]]


def test_attention_by_hand():
    P, D = 16, 64
    codes = np.zeros((2, 2, 1, P, D // 2), np.uint8)
    one = np.float32(1).view(np.uint32)
    words = np.full((2, 2, 1, P), one, np.uint32)
    # three tokens in page 1: keys 0, 1, 2 and values 3, 6, 9 in feature 0
    for t in range(3):
        codes[1, 0, 0, t, 0], codes[1, 1, 0, t, 0] = t, 3 * (t + 1)
    q = np.zeros((3, 2, D))
    q[:, 0, 0], q[:, 1, 0] = np.log(2), -np.log(2)
    table = np.array([[1, -1]], np.int32)
    o = RL.attention(q[:1], codes, words, table, [3], scale=1.0).reshape(1, 2, D)
    assert np.allclose(o[0, :, 0], [(3 + 12 + 36) / 7, (12 + 12 + 9) / 7]) and (o[..., 1:] == 0).all()
    o = RL.attention(q, codes, words, table, [3], [0, 2], scale=1.0).reshape(3, 2, D)
    assert np.allclose(o[0, :, 0], [(3 + 12) / 3, (6 + 6) / 3]) and np.allclose(o[1, 0, 0], 51 / 7) and np.isnan(o[2]).all()
    # a query in front of the first key; a page that is not there
    assert (RL.attention(q[:2], codes, words, table, [1], [0, 2])[0] == 0).all()
    assert (RL.attention(q[:1], codes, words, np.array([[2]], np.int32), [3]) == 0).all()


def test_planted_mistakes_are_caught(monkeypatch):
    def caught(test, name, wrong):
        with monkeypatch.context() as m:
            m.setattr(RL, name, wrong)
            with pytest.raises(AssertionError):
                test()
    norm, rope, hold, values, attention = RL.norm, RL.rope, RL.hold, RL.values, RL.attention
    caught(test_norm_by_hand, "norm", lambda X, W, R=None, eps=0, rounded=None: norm(X, W, R, 0))
    caught(test_norm_by_hand, "norm", lambda X, W, R=None, eps=0, rounded=None: norm(X, np.ones(4), R, eps))
    caught(test_swiglu_by_hand, "swiglu", lambda G: (lambda g, u: g * u / (1 + np.exp(-u)))(*np.split(np.asarray(G, float), 2, 1)))
    caught(test_rope_by_hand, "rope", lambda x, p, f, parts, i=False: rope(x, -np.asarray(p), f, parts, i))
    caught(test_rope_by_hand, "rope", lambda x, p, f, parts, i=False: rope(x, p, f, parts))
    caught(test_rope_by_hand, "rope", lambda x, p, f, parts, i=False: rope(x, np.float32(p), f, parts, i))
    caught(test_held_by_hand, "hold", lambda x: (lambda c, w: (c, w & ~np.uint32(15)))(*hold(x)))
    caught(test_held_by_hand, "hold", lambda x: hold(np.abs(x)))
    caught(test_held_by_hand, "packed", lambda c: (16 * c[..., 0::2] + c[..., 1::2]).astype(np.uint8))
    caught(test_attention_by_hand, "attention", lambda q, c, w, t, n, cu=None, scale=None: attention(q, c[:, ::-1], w, t, n, cu, scale))
    caught(test_attention_by_hand, "attention", lambda q, c, w, t, n, cu=None, scale=None: attention(q, c, w, t, np.asarray(n) + 1, cu, scale))


# ---------------------------------------------------------------- refusals

def norm(X=FAKE, R=None, t=0, M=4, H=128, W=FAKE, wt=0, eps=1e-6, h=None, Y=None, q=FAKE, s=FAKE):
    return B.lib().aq_norm_quant(X, R, t, M, H, W, wt, eps, h, Y, q, s, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), -2), (dict(M=(1 << 20) + 1), -2), (dict(H=0), -2), (dict(H=96), -2), (dict(H=32832), -2), (dict(t=3), -8),
    (dict(wt=-1), -8), (dict(eps=-1e-9), -8), (dict(eps=float("nan")), -8), (dict(eps=float("inf")), -8),
    (dict(X=None), -1), (dict(W=None), -1), (dict(q=None), -1), (dict(s=None), -1),
    (dict(X=FAKE + 4), -5), (dict(R=FAKE + 8), -5), (dict(W=FAKE + 2), -5), (dict(h=FAKE + 4), -5), (dict(Y=FAKE + 4), -5),
    (dict(q=FAKE + 8), -5), (dict(s=FAKE + 2), -5),
    (dict(h=FAKE + 512), -8), (dict(R=FAR, h=FAR + 16), -8), (dict(R=FAR, h=FAR - 16), -8),   # h half over X or R
])
def test_norm_refused(aqlib, over, code):
    assert norm(**over) == code


def swiglu(GU=FAKE, ld=256, M=4, I=128, Y=None, q=FAKE, s=FAKE):
    return B.lib().aq_swiglu_quant(GU, ld, M, I, Y, q, s, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), -2), (dict(M=1 << 21), -2), (dict(I=0), -2), (dict(I=100), -2), (dict(I=32832, ld=1 << 17), -2), (dict(ld=252), -2),
    (dict(ld=258), -2), (dict(ld=(1 << 22) + 4), -2), (dict(GU=None), -1), (dict(q=None), -1), (dict(s=None), -1),
    (dict(GU=FAKE + 4), -5), (dict(Y=FAKE + 4), -5), (dict(q=FAKE + 4), -5), (dict(s=FAKE + 1), -5),
])
def test_swiglu_refused(aqlib, over, code):
    assert swiglu(**over) == code


def kv4(**over):
    d = dict(pages=4, tokens=16, heads=2, D=128, codes=FAKE, words=FAKE)
    d.update(over)
    return ctypes.byref(B.AqKv4(**d))


CACHES = [(dict(pages=0), -2), (dict(tokens=8), -2), (dict(tokens=48), -2), (dict(tokens=512), -2), (dict(heads=0), -2),
          (dict(heads=1025), -2), (dict(D=96), -2), (dict(D=256), -2), (dict(codes=None), -1), (dict(words=None), -1),
          (dict(codes=FAKE + 8), -5), (dict(words=FAKE + 4), -5)]


def ropes(axes=2, part=(40, 24), pairs=64, freq=FAKE, interleaved=0):
    return ctypes.byref(B.AqRope(pairs, interleaved, axes, (ctypes.c_int32 * 4)(*part), freq))


def append(qkv=FAKE, ldqkv=1024, M=4, Hq=4, rope=None, pos=FAKE, cache=None, slots=FAKE, Q=FAR, ldq=512):
    return B.lib().aq_rope_kv4(qkv, ldqkv, M, Hq, ropes() if rope is None else rope, pos, cache or kv4(), slots, Q, ldq, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), -2), (dict(M=1 << 21), -2), (dict(Hq=-1), -2), (dict(Hq=8193), -2), (dict(ldqkv=1020), -2), (dict(ldqkv=1026), -2),
    (dict(ldqkv=1 << 23), -2), (dict(ldq=508), -2), (dict(ldq=514), -2),
    (dict(rope=ropes(axes=0)), -2), (dict(rope=ropes(axes=5)), -2), (dict(rope=ropes(part=(40, 25))), -2),
    (dict(rope=ropes(part=(70, -6))), -2), (dict(rope=ropes(pairs=65, part=(40, 25))), -2), (dict(rope=ropes(pairs=0, part=(0, 0))), -2),
    (dict(rope=ropes(freq=None)), -1), (dict(pos=None), -1), (dict(qkv=None), -1), (dict(slots=None), -1), (dict(Q=None), -1),
    (dict(qkv=FAKE + 4), -5), (dict(Q=FAR + 4), -5), (dict(slots=FAKE + 4), -5), (dict(pos=FAKE + 2), -5), (dict(rope=ropes(freq=FAKE + 1)), -5),
    (dict(Q=FAKE), -8), (dict(Q=FAKE + 2048), -8), (dict(Q=FAKE - 16), -8),      # in place at another stride; half over qkv
])
def test_append_refused(aqlib, over, code):
    assert append(**over) == code


@pytest.mark.parametrize("over,code", CACHES)
def test_caches_refused(aqlib, over, code):
    assert append(cache=kv4(**over), ldqkv=1 << 20, ldq=1 << 20) == code
    assert B.lib().aq_kv4_read(kv4(**over), FAKE, 4, FAKE, FAKE, None) == code
    assert attn(cache=kv4(**over)) == code
    assert B.lib().aq_attn_kv4_workspace_bytes(kv4(**over), 4, 4, 8, 1 << 12) == 0


def test_read_refused(aqlib):
    read = lambda M=4, s=FAKE, K=FAKE, V=FAKE: B.lib().aq_kv4_read(kv4(), s, M, K, V, None)  # noqa: E731
    assert [read(M=-1), read(M=1 << 21), read(s=None), read(K=None), read(V=None), read(s=FAKE + 4), read(K=FAKE + 8),
            read(V=FAKE + 4)] == [-2, -2, -1, -1, -1, -5, -5, -5]


def attn(Q=FAKE, ldq=512, M=4, Hq=4, cache=None, table=FAKE, width=8, kv_len=FAKE, cu=None, B_=4, scale=0.1, out=FAR, ws=FAKE, n=1 << 40):
    return B.lib().aq_attn_kv4(Q, ldq, M, Hq, cache or kv4(), table, width, kv_len, cu, B_, scale, out, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1, B_=1, cu=FAKE), -2), (dict(M=(1 << 20) + 1, cu=FAKE), -2), (dict(B_=0, cu=FAKE), -2), (dict(B_=1 << 21, cu=FAKE), -2),
    (dict(Hq=3, ldq=384), -2), (dict(Hq=0), -2), (dict(Hq=8194, ldq=1 << 21), -2), (dict(M=1 << 20, B_=1 << 20, Hq=2048, ldq=1 << 19), -2),
    (dict(width=0), -2), (dict(width=1 << 27), -2), (dict(ldq=508), -2), (dict(ldq=514), -2), (dict(ldq=1 << 23), -2),
    (dict(scale=float("nan")), -8), (dict(scale=-1.0), -8), (dict(scale=float("inf")), -8), (dict(M=3), -8),
    (dict(Q=None), -1), (dict(table=None), -1), (dict(kv_len=None), -1), (dict(out=None), -1),
    (dict(Q=FAKE + 8), -5), (dict(out=FAR + 4), -5), (dict(table=FAKE + 2), -5), (dict(kv_len=FAKE + 1), -5), (dict(cu=FAKE + 3), -5),
    (dict(out=FAKE), -8), (dict(out=FAKE + 4096), -8), (dict(out=FAKE - 4096), -8),
    (dict(width=1 << 12, ws=None), -6), (dict(width=1 << 12, n=64), -6), (dict(width=1 << 12, ws=FAKE + 8), -5),
])
def test_attention_refused(aqlib, over, code):
    assert attn(**over) == code


def test_nothing_to_do(aqlib):
    assert norm(M=0, X=None, W=None, q=None, s=None) == 0 and swiglu(M=0, GU=None) == 0
    assert append(M=0, qkv=None, Q=None) == 0 and B.lib().aq_kv4_read(kv4(), None, 0, None, None, None) == 0
    assert attn(M=0, cu=FAKE, Q=None, out=None) == 0
    assert norm(M=0, H=96) == -2 and attn(M=0, cu=FAKE, width=0) == -2
    assert B.lib().aq_attn_kv4_workspace_bytes(kv4(), 0, 4, 4, 1 << 12) == 0


def test_workspace_grows_with_ranges_only(aqlib):
    size = lambda M, B_, Hq, width: B.lib().aq_attn_kv4_workspace_bytes(kv4(tokens=64), M, B_, Hq, width)  # noqa: E731
    # one range: two units of keys, or row tiles that fill the chip by themselves
    assert size(1, 1, 8, 1) == size(1, 1, 8, 8) == size(1 << 17, 1, 16, 1 << 12) == 0
    # at most 64 ranges a tile, whatever the table's width, and a number of them in all that does not grow with the batch
    assert 0 < size(1, 1, 8, 16) < size(1, 1, 8, 1 << 14) == size(1, 1, 8, 1 << 20)
    packed = lambda n: (2 * n + 64 + 1) * 16 * 132 * 4 * 2 + 4 * (4 + 2 * n)   # noqa: E731  (2 heads; rows of 16 at most; the index)
    assert size(128, 128, 8, 1 << 14) <= packed(128)
    # by number, beyond 128 single tokens, as many ranges as make 8192 with the heads: 8192 x 4 rows x 132 values
    assert size(256, 256, 8, 1 << 14) <= max(packed(256), 8192 * 4 * 132 * 4)


def test_binding_refuses(aqlib):
    z = torch.zeros
    for f in (lambda: B.aq_norm_quant(z(2, 64), z(64)), lambda: B.aq_swiglu_quant(z(2, 128)), lambda: B.aq_rope_axes(z(32), (32,), 64),
              lambda: B.aq_kv4_cache(2, 16, 1, 64, device="cpu"), lambda: B.aq_kv4_cache_of(z(2), z(2)),
              lambda: B.aq_attn_kv4(z(2, 1, 64), None, None, None)):
        with pytest.raises(ValueError):
            f()
    for parts in ((), (1,) * 5, (40,), (-1, 4), (0,)):
        with pytest.raises(ValueError):
            B.aq_rope_axes(z(32), parts, 64)


def test_handles_are_frozen(aqlib):
    """The calls pass the descriptor made with the handle: another tensor in its
    place would leave the kernels with the old one's memory."""
    r = B.Rope(torch.zeros(32), (20, 12), 64, False)
    assert r.desc.pairs == 32 and list(r.desc.part) == [20, 12, 0, 0] and r.desc.freq == r.freq.data_ptr()
    for name in ("freq", "parts", "D", "interleaved"):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(r, name, None)
    assert dataclasses.replace(r, parts=(32,)).desc.axes == 1


# ---------------------------------------------------------------- sanitizers

@pytest.mark.timeout(600)
def test_host_file_under_asan_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "layer_host_check")
    src = [os.path.join(ROOT, "mixed_precision_int_amd", "csrc", "aq_layer_api.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "layer_host_check.cpp")]
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), *src, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0"))
    assert r.returncode == 0 and "layer host check: ok" in r.stdout, (r.stdout[-4000:], r.stderr[-4000:])
