"""Host side of the per-token-factor operators beside test_routed_cpu.py: what
a caller does with the packed experts and the adapters between calls."""
import dataclasses

import numpy as np
import pytest
import torch

from mixed_precision_int_amd import binding as B


def adapters(L=2, R=8, K=64, N=64):
    """A pool on the host (never passed to a call)."""
    A, Bm = torch.zeros(L, R, K), torch.zeros(L, N, R)
    sc, ranks = torch.ones(L), torch.full((L,), R, dtype=torch.int32)
    d = B.AqLora(L, R, K, N, B.AQ_TYPE_F32, A.data_ptr(), Bm.data_ptr(), sc.data_ptr(), ranks.data_ptr())
    return B.LoraAdapters(A, Bm, sc, ranks, d)


def experts(E=2, H=128, I=128):
    def packed(N, K):
        labels = B.aq_labels_from_map(np.full((N // 64, K // 128), 8, np.uint8))
        return B.aq_alloc_packed(B.aq_plan_pack(N, K, 64, 128, labels), labels, device="cpu")
    return B.PackedExperts(packed(E * 2 * I, H), packed(E * H, I), E)


def test_pools_do_not_take_other_tensors(aqlib):
    """The calls pass the descriptor made with the pool: another tensor in its
    place would leave the kernels with the old one's memory."""
    pool, ex = adapters(), experts()
    for name in ("A", "B", "scale", "ranks", "desc"):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(pool, name, getattr(pool, name))
    for name in ("gate_up", "down", "E"):
        with pytest.raises(dataclasses.FrozenInstanceError):
            setattr(ex, name, getattr(ex, name))


def test_pools_remade(aqlib):
    """A pool remade with another part has a descriptor of its own, or is refused
    where the descriptor is given and names another tensor."""
    pool, ex, other = adapters(), experts(), experts()
    new = dataclasses.replace(ex, down=other.down)
    assert new._desc[1]._obj.w8 == other.down.w8.data_ptr() and ex._desc[1]._obj.w8 == ex.down.w8.data_ptr()
    assert B.aq_moe_workspace_bytes(new, 4, 2) == B.aq_moe_workspace_bytes(ex, 4, 2) > 0
    dataclasses.replace(pool)
    for name in ("A", "B", "scale", "ranks"):
        with pytest.raises(ValueError):
            dataclasses.replace(pool, **{name: getattr(pool, name).clone()})
    for name in ("scale", "ranks"):
        with pytest.raises(ValueError):
            dataclasses.replace(pool, **{name: None})
