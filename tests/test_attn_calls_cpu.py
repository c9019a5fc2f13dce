"""Calls of the attention over the 4-bit cache that launch nothing, beside those of test_layer_cpu.py."""
import pytest

from mixed_precision_int_amd import binding as B
from tests.test_layer_cpu import FAKE, attn, kv4


def test_no_sequences(aqlib):
    """An empty batch is a no-op like every other empty call; rows without sequences are refused."""
    assert attn(M=0, B_=0, cu=FAKE, Q=None, table=None, kv_len=None, out=None) == 0 and attn(M=0, B_=0, Q=None, out=None) == 0
    assert B.lib().aq_attn_kv4_workspace_bytes(kv4(), 0, 0, 4, 8) == 0
    assert attn(M=1, B_=0, cu=FAKE) == -2 and attn(M=0, B_=-1, cu=FAKE) == -2


@pytest.mark.parametrize("scale,code", [(0.0, 0), (2.0 ** 127, 0), (1.8e38, -8), (3.4e38, -8)])
def test_scales_past_the_range_refused(aqlib, scale, code):
    """The scale in powers of two, scale * log2(e), has to be an FP32 number: past it every row would be NaN."""
    assert attn(M=0, B_=0, scale=scale) == code and (code == 0 or attn(scale=scale) == code)
