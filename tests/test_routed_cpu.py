"""The per-token-factor operators without a GPU: the oracle pinned to
hand-worked cases, the library's refusals (every one before a launch), and
its host file under AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from mixed_precision_int_amd import binding as B
from oracle import aq_oracle as O
from oracle import routed as RO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # 16-byte-aligned fake device address; never dereferenced


# ---------------------------------------------------------------- oracle

def test_route_by_hand():
    X = np.array([[1.0, 0.0], [0.0, 1.0]])
    W = np.log(np.array([[1, 8], [2, 1], [4, 1], [1, 8]], dtype=np.float64))
    ids, w = RO.route(X, W, 2)
    # token 0: shares 1 2 4 1 of 8; token 1: 8 1 1 8 of 18, the tie to expert 0
    assert ids.tolist() == [[2, 1], [0, 3]]
    assert np.allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]], rtol=1e-14)
    _, w = RO.route(X, W, 2, norm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5], [16 / 18, 16 / 18]], rtol=1e-14)
    # sigmoid(log x) = x / (1 + x); the bias moves the choice, not the weight
    ids, w = RO.route(X, W, 2, bias=[1.0, 0.0, 0.0, 0.0], score="sigmoid", norm=False)
    assert ids.tolist() == [[0, 2], [0, 3]]
    assert np.allclose(w, [[1 / 2, 4 / 5], [8 / 9, 8 / 9]], rtol=1e-14)
    # excluded experts; fewer left than slots
    ids, w = RO.route(X, W, 3, bias=[-np.inf, 0.0, -np.inf, -np.inf])
    assert ids.tolist() == [[1, -1, -1]] * 2 and w.tolist() == [[1.0, 0.0, 0.0]] * 2


def test_lora_by_hand():
    Y, X = np.zeros((3, 2)), np.array([[1.0, 2.0], [1.0, 2.0], [3.0, 0.0]])
    A = np.array([[[1.0, 1.0], [5.0, 5.0]], [[0.0, 1.0], [1.0, 0.0]]])      # [L, R, K]
    Bm = np.array([[[1.0, 7.0], [2.0, 7.0]], [[1.0, 1.0], [0.0, 2.0]]])     # [L, N, R]
    out, mag = RO.lora(Y, X, [0, -1, 1], A, Bm, scale=[2.0, 1.0], ranks=[1, 2])
    assert out.tolist() == [[6.0, 12.0], [0.0, 0.0], [3.0, 6.0]]
    assert mag.tolist() == out.tolist()


def test_experts_against_dequantized_weights():
    """The experts' definition equals plain matrix products with the
    dequantized weights, up to the order of FP64 sums, and a slot that holds
    no expert adds nothing."""
    rng = np.random.default_rng(2)
    E, H, I, M, k = 3, 128, 64, 4, 2
    W13 = rng.standard_normal((E * 2 * I, H)).astype(np.float32) * 0.1
    W2 = rng.standard_normal((E * H, I)).astype(np.float32) * 0.1
    gu = O.quant_weights(W13, rng.choice([4, 8], size=(E * 2 * I // 64, 1)), 64, 128)
    dn = O.quant_weights(W2, rng.choice([4, 8], size=(E * H // 64, 1)), 64, 64)
    X = rng.standard_normal((M, H)).astype(np.float32)
    q, s = O.quant_act(X)
    ids = np.array([[0, 2], [1, -1], [2, 2], [5, 0]])
    w = rng.random((M, k)).astype(np.float32)
    Y, mag = RO.experts(q, s, ids, w, gu, dn, E, (128, 64))
    D13 = (gu[0] * np.repeat(gu[1].astype(np.float64), 128, 1)).reshape(E, 2 * I, H)
    D2 = (dn[0] * np.repeat(dn[1].astype(np.float64), 64, 1)).reshape(E, H, I)
    for m in range(M):
        y = np.zeros(H)
        for i in range(k):
            e = ids[m, i]
            if not 0 <= e < E:
                continue
            g, u = np.split(D13[e] @ (q[m] * np.float64(s[m])), 2)
            h = (g / (1 + np.exp(-g)) * u).astype(np.float32)
            qh, sh = O.quant_act(h[None])
            y += w[m, i] * (D2[e] @ (qh[0] * np.float64(sh[0])))
        assert np.abs(Y[m] - y).max() <= 1e-12 * np.abs(y).max()
        assert (mag[m] >= np.abs(Y[m]) * (1 - 1e-12)).all()


def test_planted_mistakes_are_caught(monkeypatch):
    """The pins above fail for: ties to the last expert, weights with the bias
    in them, ranks beyond an adapter's, up and gate exchanged."""
    real_route, real_lora, real_linear = RO.route, RO.lora, RO.linear64

    def last_tie(X, Wr, top_k, *a, **k):
        ids, w = real_route(X, np.asarray(Wr)[::-1], top_k, *a, **k)
        return np.where(ids >= 0, len(Wr) - 1 - ids, ids), w

    def biased(X, Wr, top_k, bias=None, **k):
        ids, w = real_route(X, Wr, top_k, bias, **k)
        return ids, w if bias is None else w + np.asarray(bias)[ids]

    for wrong in (last_tie, biased):
        monkeypatch.setattr(RO, "route", wrong)
        with pytest.raises(AssertionError):
            test_route_by_hand()
    monkeypatch.setattr(RO, "lora", lambda Y, X, ids, A, Bm, scale=None, ranks=None: real_lora(Y, X, ids, A, Bm, scale))
    with pytest.raises(AssertionError):
        test_lora_by_hand()

    def swapped(qx, sx, codes, sW, bK):
        y, a = real_linear(qx, sx, codes, sW, bK)
        return (np.roll(y, y.shape[1] // 2, 1), a) if bK == 128 else (y, a)
    monkeypatch.setattr(RO, "linear64", swapped)
    with pytest.raises(AssertionError):
        test_experts_against_dequantized_weights()


# ---------------------------------------------------------------- refusals

def packed(N, K, bK=128, **over):
    T = (N // 64) * (K // bK)
    d = B.AqPacked(N, K, 64, bK, T // 2, T - T // 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def route(X=FAKE, M=4, K=128, Wr=FAKE, wt=0, E=16, bias=None, k=2, score=0, norm=1, scale=1.0, ids=FAKE, w=FAKE,
          ws=FAKE, n=1 << 30):
    return B.lib().aq_moe_route(X, M, K, Wr, wt, E, bias, k, score, norm, scale, ids, w, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), -2), (dict(K=0), -2), (dict(K=96), -2), (dict(K=1 << 23), -2), (dict(M=(1 << 20) + 1), -2),
    (dict(E=0), -2), (dict(E=1025), -2), (dict(k=0), -8), (dict(k=17), -8), (dict(E=64, k=33), -8), (dict(wt=2), -8),
    (dict(score=2), -8), (dict(scale=float("inf")), -8), (dict(scale=float("nan")), -8),
    (dict(X=None), -1), (dict(Wr=None), -1), (dict(ids=None), -1), (dict(w=None), -1),
    (dict(X=FAKE + 4), -5), (dict(Wr=FAKE + 8), -5), (dict(ids=FAKE + 1), -5), (dict(w=FAKE + 2), -5),
    (dict(bias=FAKE + 2), -5), (dict(ws=None), -6), (dict(n=4 * 16 * 8 - 1), -6), (dict(ws=FAKE + 4), -5),
])
def test_route_refused(aqlib, over, code):
    assert route(**over) == code


def test_route_no_tokens(aqlib):
    assert route(M=0, X=None, ws=None) == 0
    assert aqlib.aq_moe_route_workspace_bytes(0, 128, 16) == 0
    assert aqlib.aq_moe_route_workspace_bytes(4, 100, 16) == 0
    assert aqlib.aq_moe_route_workspace_bytes(4, 128, 2000) == 0
    # the largest call's logits: one FP64 value per token and expert at least
    assert aqlib.aq_moe_route_workspace_bytes(1024, 5120, 160) >= 8 * 1024 * 160


E, H, I = 6, 256, 128


def experts(gu=None, dn=None, E=E, qx=FAKE, sx=FAKE, M=4, ids=FAKE, w=FAKE, k=2, Y=FAKE, ws=FAKE, n=1 << 40):
    gu = packed(6 * 2 * I, H) if gu is None else gu
    dn = packed(6 * H, I) if dn is None else dn
    return B.lib().aq_moe_experts(ctypes.byref(gu), ctypes.byref(dn), E, qx, sx, M, ids, w, k, Y, ws, n, None)


def layer(gu=None, dn=None, E=E, X=FAKE, M=4, Wr=FAKE, wt=1, bias=None, k=2, score=1, scale=1.0, ids=FAKE, w=FAKE,
          Y=FAKE, ws=FAKE, n=1 << 40):
    gu = packed(6 * 2 * I, H) if gu is None else gu
    dn = packed(6 * H, I) if dn is None else dn
    return B.lib().aq_moe_layer(ctypes.byref(gu), ctypes.byref(dn), E, X, M, Wr, wt, bias, k, score, 1, scale, ids, w, Y,
                                ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(E=0), -2), (dict(E=5), -2), (dict(E=2000), -2), (dict(M=-1), -2), (dict(M=(1 << 20) + 1), -2), (dict(k=0), -8),
    (dict(k=33), -8), (dict(gu=packed(6 * 2 * I, 2 * H)), -2), (dict(dn=packed(6 * H, 2 * I)), -2),
    (dict(gu=packed(6 * 2 * I, H, T4=3)), -4), (dict(dn=packed(6 * H, I, w8=None)), -1),
    (dict(dn=packed(6 * H, I, bN=32)), -3), (dict(gu=packed(6 * 2 * I, H, labels=FAKE + 2)), -5),
    (dict(Y=None), -1), (dict(Y=FAKE + 4), -5), (dict(ids=None), -1), (dict(w=FAKE + 1), -5),
    (dict(ws=None), -6), (dict(n=100), -6), (dict(ws=FAKE + 8), -5),
])
def test_experts_and_layer_refused(aqlib, over, code):
    assert experts(**over) == code
    assert layer(**over) == code


def test_experts_and_layer_refused_apart(aqlib):
    assert experts(qx=None) == -1 and experts(qx=FAKE + 8) == -5 and experts(sx=None) == -1
    assert layer(X=None) == -1 and layer(X=FAKE + 8) == -5 and layer(Wr=None) == -1 and layer(wt=2) == -8
    assert layer(k=7) == -8 and layer(score=3) == -8 and layer(scale=float("nan")) == -8
    # more slots than experts are a router's error, not the experts' part's
    assert experts(k=7, n=0) == -6
    assert experts(M=0, qx=None, ws=None) == 0 and layer(M=0, X=None, ws=None) == 0
    lib, gu, dn = B.lib(), packed(6 * 2 * I, H), packed(6 * H, I)
    n = [lib.aq_moe_workspace_bytes(ctypes.byref(gu), ctypes.byref(dn), 6, m, 2) for m in (0, 1, 4, 64, 1024, 1 << 20, (1 << 20) + 1)]
    assert n[0] == n[6] == 0 and 0 < n[1] < n[2] < n[3] < n[4] < n[5]
    assert lib.aq_moe_workspace_bytes(ctypes.byref(gu), ctypes.byref(dn), 7, 4, 2) == 0
    assert experts(n=n[2] - 1) == -6 and layer(n=n[2] - 1) == -6


def lora(over=None, X=FAKE, M=4, ids=FAKE, Yin=FAKE, ldyin=128, Y=FAKE, ldy=128, ws=FAKE, n=1 << 40):
    ad = B.AqLora(3, 16, 256, 128, 1, FAKE, FAKE, FAKE, FAKE)
    for k, v in (over or {}).items():
        setattr(ad, k, v)
    return B.lib().aq_lora_add(ctypes.byref(ad), X, M, ids, Yin, ldyin, Y, ldy, ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(L=0), -2), (dict(L=8193), -2), (dict(R=0), -2), (dict(R=12), -2), (dict(R=136), -2), (dict(K=100), -2),
    (dict(N=96), -2), (dict(N=1 << 21), -2), (dict(K=1 << 21), -2), (dict(type=3), -8), (dict(type=-1), -8),
    (dict(A=None), -1), (dict(B=None), -1), (dict(A=FAKE + 8), -5), (dict(B=FAKE + 2), -5), (dict(scale=FAKE + 1), -5),
    (dict(rank=FAKE + 2), -5),
])
def test_lora_descriptor_refused(aqlib, over, code):
    assert lora(over) == code


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), -2), (dict(M=(1 << 20) + 1), -2), (dict(X=None), -1), (dict(ids=None), -1), (dict(Yin=None), -1),
    (dict(Y=None), -1), (dict(X=FAKE + 4), -5), (dict(ids=FAKE + 1), -5), (dict(Yin=FAKE + 4), -5), (dict(Y=FAKE + 8), -5),
    (dict(ldy=64), -2), (dict(ldyin=64), -2), (dict(ldy=130), -2), (dict(ldyin=(1 << 22) + 4), -2),
    (dict(ldy=256), -8),                       # in place at another stride
    (dict(Y=FAKE + 64), -8),                   # overlapping
    (dict(Y=FAKE + 4 * 3 * 128 + 4 * 112), -8),
    (dict(ws=None), -6), (dict(n=64), -6), (dict(ws=FAKE + 4), -5),
])
def test_lora_call_refused(aqlib, over, code):
    assert lora(**over) == code


def test_lora_no_tokens_and_workspace(aqlib):
    assert lora(M=0, X=None, ws=None) == 0
    ad = B.AqLora(3, 16, 4096, 4096, 1, FAKE, FAKE, None, None)
    n = [aqlib.aq_lora_workspace_bytes(ctypes.byref(ad), m) for m in (0, 1, 64, 8192)]
    assert n[0] == 0 and 0 < n[1] < n[2] < n[3]
    ad.R = 20
    assert aqlib.aq_lora_workspace_bytes(ctypes.byref(ad), 4) == 0


def test_binding_refuses_host_tensors():
    import torch
    X, W = torch.zeros(2, 128), torch.zeros(4, 128)
    with pytest.raises(ValueError):
        B.aq_moe_route(X, W, 2)
    with pytest.raises(ValueError):
        B.aq_lora_adapters(torch.zeros(1, 8, 128), torch.zeros(1, 64, 8))


# ---------------------------------------------------------------- sanitizers

@pytest.mark.timeout(600)
def test_host_file_under_asan_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "routed_host_check")
    src = [os.path.join(ROOT, "mixed_precision_int_amd", "csrc", "aq_routed_api.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "routed_host_check.cpp")]
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), *src, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0"))
    assert r.returncode == 0 and "routed host check: ok" in r.stdout, (r.stdout[-4000:], r.stderr[-4000:])
