"""Two steps of a decoder captured on one stream, of sizes whose projections cut their input columns between
workgroups, replayed side by side: neither's sums reach the other's, nor do a larger eager step's."""
import numpy as np
import pytest
import torch

import mixed_precision_int_amd as aq
import mixed_precision_int_amd.model as mdl
from tests.parity import to_dev
from tests.test_gpu_layer import freqs

pytestmark = pytest.mark.gpu

H, I, HEADS, KV, D, LAYERS, P = 256, 4096, 4, 2, 64, 2, 16
GEOMETRY = [("qkv", (HEADS + 2 * KV) * D, H), ("o", H, HEADS * D), ("gate_up", 2 * I, H), ("down", H, I)]


def test_captured_steps_have_their_own_workspace():
    rng = np.random.default_rng(17)
    maps = [[rng.choice([4, 8], size=(N // 64, K // 128)) for _, N, K in GEOMETRY] for _ in range(LAYERS)]
    model = mdl.pack_model(GEOMETRY, maps, lambda l, name, N, K: to_dev((rng.standard_normal((N, K)) * 0.05).astype(np.float32)))
    norm = lambda: to_dev((rng.random(H) + 0.5).astype(np.float32))  # noqa: E731
    dec = mdl.Decoder(model, [norm() for _ in range(LAYERS)], [norm() for _ in range(LAYERS)], norm(),
                      aq.aq_rope_axes(to_dev(freqs(D // 2, 1e4)), (D // 2,), D), HEADS, KV, D)
    sizes = (36, 48, 64)
    assert all(dec.workspace(B, torch.device("cuda", 0)).numel() > mdl.COUNTER_BYTES for B in sizes)

    def inputs(B):
        table = torch.randperm(2 * B, device="cuda").int().view(B, 2)
        pos = torch.randint(0, 2 * P, (B,), device="cuda").int()
        slots = table.gather(1, (pos // P).long()[:, None])[:, 0].long() * P + pos % P
        caches = dec.caches(2 * B, P)
        for c in caches:
            c.codes.random_(0, 256)
            c.words.copy_((torch.rand(c.words.shape, device="cuda") + 0.5).view(torch.int32) & ~15 | 7)
        return torch.randn((B, H), device="cuda"), caches, pos, slots, table, pos + 1

    given = [inputs(B) for B in sizes]
    want = [[t.clone() for t in dec.step(*a)] for a in given]
    capture, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    with torch.cuda.stream(capture):
        for a in given[:2]:
            dec.step(*a)
            capture.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=capture):
                outs = dec.step(*a)
            graphs.append((g, outs, torch.cuda.Stream()))
    for _ in range(6):
        for _, outs, _ in graphs:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(capture):
            big = dec.step(*given[2])
        eager = [dec.step(*a) for a in given[:2]]
        torch.cuda.synchronize()
        for got, ref in zip([g[1] for g in graphs] + [big] + eager, want[:2] + want[2:] + want[:2]):
            for x, y in zip(got, ref):
                assert torch.equal(x, y)
