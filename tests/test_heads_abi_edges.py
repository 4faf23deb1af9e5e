"""Host-side tests of the operators on heads and groups: descriptors whose
numbers are finite and whose results would be none.  No GPU is used."""
import pytest

from test_heads_abi import rotary
from test_seq_abi import BAD, _refused


@pytest.mark.parametrize("kw", [
    dict(amplitude=1e39), dict(amplitude=-1e300),                                    # no fp32 number
    dict(scaling="linear", factor=1e-310), dict(scaling="parts", factor=1e-310, original=4096, amplitude=1.0),
    dict(scaling="base", factor=1e-300),                                             # theta underflows, frequencies overflow
    dict(theta=1e-320, d=256), dict(theta=1e-305, d=256),                                   # turns of far positions overflow
])
def test_rotary_of_no_numbers_is_refused(kw):
    _refused(rotary, BAD, **kw)


@pytest.mark.parametrize("kw", [dict(amplitude=3e38), dict(amplitude=0.0), dict(scaling="linear", factor=1e-6),
                                dict(scaling="base", factor=1e200), dict(theta=1e-3), dict(theta=1e300)])
def test_rotary_of_large_numbers_is_taken(kw):
    rotary(**kw).close()
