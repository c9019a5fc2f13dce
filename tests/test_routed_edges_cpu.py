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


@pytest.mark.parametrize("change,text", [
    (dict(gate=lambda a: a.bfloat16(), up=lambda a: a.bfloat16(), down=lambda a: a.bfloat16()), "float32"),
    (dict(gate=lambda a: a.double()), "float32"), (dict(down=lambda a: a.half()), "float32"),
    (dict(map_gate_up=lambda z: z[:-1]), "map_gate_up"), (dict(map_gate_up=lambda z: z.T), "map_gate_up"),
    (dict(map_gate_up=lambda z: z.reshape(-1)), "map_gate_up"), (dict(map_down=lambda z: z[:, :1]), "map_down"),
    (dict(map_down=lambda z: z[:1]), "map_down"), (dict(up=lambda a: a[:1]), "up"), (dict(gate=lambda a: a[0]), "gate"),
    (dict(), "device"),
])
def test_pack_experts_refused(monkeypatch, change, text):
    """Weights of another type and maps of another shape are refused before the
    packer reads either."""
    from mixed_precision_int_amd import model
    packed = []

    def pack(W, labels, bN, bK):
        packed.append(W)
        raise RuntimeError("packed")
    monkeypatch.setattr(model, "aq_pack_weights", pack)
    E, I, H = 3, 256, 256
    a = dict(gate=torch.zeros(E, I, H), up=torch.zeros(E, I, H), down=torch.zeros(E, H, I),
             map_gate_up=np.full((E * 2 * I // 64, H // 128), 8, np.uint8), map_down=np.full((E * H // 64, I // 128), 4, np.uint8))
    for k, f in change.items():
        a[k] = f(a[k])
    with pytest.raises(ValueError, match=text):
        model.pack_experts(**a)
    assert not packed
