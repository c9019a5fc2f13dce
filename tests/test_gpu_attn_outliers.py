"""Queries with a feature far larger than the others, and queries far from zero, over keys that take those
out of the scores: what is left of q is then what the scores are made of, and no kernel may have lost it.

The tolerances are test_gpu_layer.py's.  q enters the kernel for few rows as whole numbers of its row's largest value, rounded at
2^-30 of it, products and the zero point's share exact, so a score is off by at most 2^-30 scale max|q| sum|k|.  Here
max|q| < 2^10 and the other features are of size 1, so that is 2^-20 scale sum|k|, which the (2D + 8) u = 2^-16 and 2^-17 of the sum
of |q||k| hold.  In norm: features are off by 2^-21 of a feature of size 1 on average, either way, and so is a score of its
size, 5e-7, inside the 2e-6.  Three digits would leave 2^8 times as much.
"""
import numpy as np
import pytest

from tests.test_gpu_layer import check_attn, filled

pytestmark = pytest.mark.gpu

# tiles of 4, 8 and 16 rows by single tokens and by packed ones; prompts
SHAPES = [dict(lens=[300, 77], new=None, Hq=8, heads=2, D=128, P=16), dict(lens=[1500], new=None, Hq=7, heads=1, D=64, P=64),
          dict(lens=[700, 5], new=None, Hq=16, heads=2, D=128, P=32), dict(lens=[400, 90], new=None, Hq=32, heads=2, D=64, P=16),
          dict(lens=[90, 300], new=None, Hq=32, heads=2, D=128, P=16), dict(lens=[300, 77], new=[3, 2], Hq=6, heads=2, D=64, P=32),
          dict(lens=[600], new=[90], Hq=8, heads=2, D=128, P=64), dict(lens=[300, 277], new=[150, 177], Hq=10, heads=2, D=128, P=64),
          dict(lens=[400, 90], new=[400, 60], Hq=5, heads=1, D=64, P=16)]


def nibbles(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def made(s, seed):
    rng = np.random.default_rng(seed)
    table, codes, words = filled(rng, s["lens"], s["P"], s["heads"], s["D"])
    cu = None if s["new"] is None else np.concatenate([[0], np.cumsum(s["new"])]).astype(np.int32)
    M = len(s["lens"]) if cu is None else int(cu[-1])
    return rng, rng.standard_normal((M, s["Hq"], s["D"])).astype(np.float32), codes, words, table, cu


@pytest.mark.parametrize("size", [30, 300])
@pytest.mark.parametrize("s", SHAPES, ids=lambda s: f"{s['new']}-{s['Hq']}-{s['D']}")
def test_one_feature_far_larger(s, size):
    rng, q, codes, words, table, cu = made(s, 41)
    ch = int(rng.integers(s["D"]))
    c = nibbles(codes)
    c[:, 0, ..., ch] = (words & 15)[:, 0]                  # every key is 0 there
    codes = (c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)
    q[..., ch] = size * (1 + rng.random(q.shape[:2]))
    check_attn(q, codes, words, table, np.array(s["lens"]), cu, name=f"outlier {size}")


@pytest.mark.parametrize("s", SHAPES[:7], ids=lambda s: f"{s['new']}-{s['Hq']}-{s['D']}")
def test_queries_far_from_zero(s):
    """Keys whose features add up to nothing under queries around 200: in whole numbers the common part leaves exactly."""
    rng, q, codes, words, table, cu = made(s, 42)
    c = nibbles(codes)
    half = c[:, 0, ..., 0::2] % 15
    c[:, 0, ..., 0::2], c[:, 0, ..., 1::2] = half, 14 - half
    words[:, 0] = words[:, 0] & ~np.uint32(15) | 7
    codes = (c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)
    check_attn(q + np.float32(200), codes, words, table, np.array(s["lens"]), cu, name="far from zero")
