"""What bench.py --decoder-step leaves out of the layers it times."""
from types import SimpleNamespace

import pytest
import torch

import bench


def test_nothing_runs_in_the_attentions_place():
    """The stand-in gives rows made before, whatever it is called with, and goes again."""
    kept = lambda *a, **k: None  # noqa: E731
    mdl, rows = SimpleNamespace(aq_attn_kv4=kept), torch.zeros(3, 8)
    q = torch.ones(3, 16).unflatten(1, (4, 4))[:, :2]          # a view of wider rows, as a layer has them
    with bench.attention_left_out(mdl, rows):
        assert mdl.aq_attn_kv4(q, None, None, None, cu_q=None) is rows
    assert mdl.aq_attn_kv4 is kept
    with pytest.raises(KeyError), bench.attention_left_out(mdl, rows):
        raise KeyError
    assert mdl.aq_attn_kv4 is kept
