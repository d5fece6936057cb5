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


class TestBinding:
    """Missing or wrong tensors raise what the block's calls raise for them, and name them."""

    x = staticmethod(lambda: pytest.importorskip("torch").zeros(2, 4, 64))

    def test_missing_pages(self):
        x = self.x()
        for call in (lambda: gdn.gdn_kv_append(x, x, None, x, x, x, None, 2, 2, 4, 64, 16, 1, 1, stream=0),
                     lambda: gdn.gdn_attn_decode(x, None, x, x, x, x, 2, 1, 4, 4, 64, 16, 1, 1, 0, 0, 1.0, x,
                                                 stream=0),
                     lambda: gdn.gdn_attn_prefill(x, None, x, x, x, x, x, 2, 2, 1, 4, 4, 64, 16, 1, 1, 0, 0,
                                                  1.0, stream=0)):
            with pytest.raises(ValueError, match="k_pages is required"):
                call()
        for call in (lambda: gdn.gdn_pages_copy(None, x, x, 1, 1, 1, 16, stream=0),
                     lambda: gdn.gdn_pages_reserve(None, x, x, x, x, 1, 16, 1, 1, 16, 1, x, stream=0),
                     lambda: gdn.gdn_pages_fork(None, x, x, x, x, x, 1, 16, 1, 1, 16, 1, 1, x, stream=0),
                     lambda: gdn.gdn_pages_compact(None, x, x, x, 16, 1, 1, 16, 1, 1, x, stream=0)):
            with pytest.raises(ValueError, match="pages is required"):
                call()

    def test_missing_rows(self):
        x = self.x()
        with pytest.raises(ValueError, match="k is required"):
            gdn.gdn_kv_append(None, x, x, x, x, x, None, 2, 2, 4, 64, 16, 1, 1, stream=0)
        with pytest.raises(ValueError, match="q is required"):
            gdn.gdn_attn_decode(None, x, x, x, x, x, 2, 1, 4, 4, 64, 16, 1, 1, 0, 0, 1.0, x, stream=0)

    def test_no_tensors(self):
        x = self.x()
        for wrong in ([1.0], 3, x.numpy()):
            with pytest.raises(TypeError, match="k_pages must be"):
                gdn.gdn_attn_decode(x, wrong, x, x, x, x, 2, 1, 4, 4, 64, 16, 1, 1, 0, 0, 1.0, x, stream=0)
            with pytest.raises(TypeError, match="pages must be"):
                gdn.gdn_pages_copy(wrong, x, x, 1, 1, 1, 16, stream=0)
