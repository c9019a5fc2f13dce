"""Calls of a decoder layer's steps beside those of test_gpu_layer.py and test_gpu_layer_edges.py."""
import pytest
import torch

import mixed_precision_int_amd as aq
from tests.test_gpu_decoder import H, LAYERS, P, decoder
from tests.test_gpu_layer import cache_of

pytestmark = pytest.mark.gpu


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("packed", [False, True])
def test_no_sequences(packed):
    cu = i32(1) if packed else None
    o = aq.aq_attn_kv4(torch.empty((0, 4, 64), device="cuda"), cache_of(2, 16, 2, 64), i32(0, 3), i32(0), cu)
    assert o.shape == (0, 256)
    dec = decoder()
    caches = dec.caches(2, P)
    qx, sx, h = dec.step(torch.empty((0, H), device="cuda"), caches, i32(0), torch.empty(0, dtype=torch.int64, device="cuda"),
                         i32(0, 3), i32(0), cu)
    assert qx.shape == h.shape == (0, H) and sx.shape == (0,) and len(caches) == LAYERS
