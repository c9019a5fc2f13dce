"""The marked activation quantizer's refusals, every one before a launch."""
import pytest

from mixed_precision_int_amd import binding as B

FAKE = 1 << 20   # 16-byte-aligned fake device address; never dereferenced


@pytest.mark.parametrize("args,code", [
    ((FAKE, 4, 100, FAKE, FAKE), -2), ((FAKE, 4, 0, FAKE, FAKE), -2), ((FAKE, -1, 128, FAKE, FAKE), -2), ((FAKE, (1 << 30) + 1, 64, FAKE, FAKE), -2),
    ((None, 4, 128, FAKE, FAKE), -1), ((FAKE, 4, 128, None, FAKE), -1), ((FAKE, 4, 128, FAKE, None), -1),
    ((FAKE + 4, 4, 128, FAKE, FAKE), -5), ((FAKE, 4, 128, FAKE + 8, FAKE), -5), ((FAKE, 4, 128, FAKE, FAKE + 2), -5),
    ((None, 0, 128, None, None), 0),
])
def test_marked_quantizer_refused(aqlib, args, code):
    assert aqlib.aq_quant_act_marked(*args, None) == code
