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


@pytest.mark.parametrize("M", [40, 100])
def test_padding_rows_change_no_other(M):
    """Rows behind the last sequence, not held (slot -1): whatever they are, the others' rows and the cache stay to the bit."""
    dec = decoder(7)
    new = [1, 20, 9]
    n, width = sum(new), 4
    table = torch.randperm(3 * width, device="cuda").int().view(3, width)
    seq = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(new, device="cuda"))
    pos = torch.cat([torch.arange(k, device="cuda") for k in new])
    slots = torch.full((M,), -1, dtype=torch.int64, device="cuda")
    slots[:n] = table[seq, pos // P].long() * P + pos % P
    positions = i32(M)
    positions[:n] = pos.int()
    lens = torch.tensor(new, device="cuda").int()
    cu = torch.tensor([0, 1, 21, 30], device="cuda").int()
    x = torch.randn((M, H), device="cuda")
    got = []
    for fill in (0.0, float("nan"), 1e30, float("inf")):
        x[n:] = fill
        caches = dec.caches(3 * width, P)
        junk = torch.full((8 << 20,), fill, device="cuda")             # (what a later allocation finds in its memory)
        del junk
        out = dec.step(x, caches, positions, slots, table, lens, cu)
        assert torch.isfinite(out[2][:n]).all() and torch.isnan(x[n:]).all() == (fill != fill)
        got.append([t[:n].clone() for t in out] + [t for c in caches for t in (c.codes, c.words)])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
