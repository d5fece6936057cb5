"""More refusals of the attention layer's calls, on the host (no GPU needed)."""
import pytest

import gated_deltanet_linear_scan_gb300 as gdn

OK, NULL, SHAPE = 0, 1, 2
P = 0x10000  # a fake device address, never dereferenced here


@pytest.fixture(scope="module")
def lib():
    gdn.build_if_needed()
    return gdn.library()


def test_selftest(lib):
    f = lib.gdn_selftest_attn_wait
    assert f(1, 1000, None, None) == NULL
    assert f(4, 1000, P, None) == SHAPE
    assert f(1, 0, P, None) == SHAPE
    assert f(1, 2000001, P, None) == SHAPE
