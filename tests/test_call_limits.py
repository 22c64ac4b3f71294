"""The largest numbers of units that calls over logits take: on the host, nothing is launched (a null pointer or a
workspace that is too small ends each accepted call)."""

import pytest

from test_pages_host import FAKE, _select, sv   # noqa: F401

LAST = (1 << 31) - (1 << 16)   # the loops over units add up to 2^16 to the last one's 32-bit number


@pytest.mark.parametrize("K,V,units", [(1, 1000, 1), (4, 2048, 4), (64, 2049, 128), (8, 1 << 20, 8 * 512)])
def test_beam_units(sv, K, V, units):   # noqa: F811
    most = (LAST - 1) // units
    assert _select(sv, B=most, K=K, V=V, logits=None) == sv.SPEC_ERR_NULL
    for B in (most + 1, ((1 << 31) - 66) // units):   # (the last would have passed the end of 32 bits on the device)
        assert _select(sv, B=B, K=K, V=V, logits=None) == sv.SPEC_ERR_SHAPE


def test_probs_units(sv):   # noqa: F811
    def call(rows, V):
        return sv.load_library().spec_probs(FAKE, 0, rows, V, 1.0, FAKE, FAKE, FAKE, 16, None)

    assert call(LAST - 1, 1000) == sv.SPEC_ERR_WORKSPACE
    assert call(LAST, 1000) == sv.SPEC_ERR_SHAPE
    assert call((1 << 31) - 66, 1000) == sv.SPEC_ERR_SHAPE
