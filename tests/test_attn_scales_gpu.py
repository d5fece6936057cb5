"""Scales that are zero or negative (every key alike, the least alike keys first), against the
plain form in 64 bits."""
import numpy as np
import pytest

from tests.attn_cases import Cache
from tests.test_attn_decode_gpu import run as decode
from tests.test_attn_prefill_gpu import run as prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("bfloat16", 64), ("float16", 128), ("bfloat16", 256), ("float32", 128)])
@pytest.mark.parametrize("scale", [0.0, -0.2])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_scales(cuda_lib, dtype, d, scale, window, sinks):
    rng = np.random.default_rng([d, window])
    lens = [400, 9, 130]
    c = Cache(torch, rng, lens, 2, d, 32, dtype)
    q = c.queries(rng, [2] * 3, 6)
    c.check(decode(cuda_lib, c, q, 2, 6, window=window, sinks=sinks, scale=scale), q, [2] * 3, scale,
            window, sinks)
    counts = [300, 9, 77]
    q = c.queries(rng, counts, 6)
    c.check(prefill(cuda_lib, c, q, counts, 6, window=window, sinks=sinks, scale=scale), q, counts, scale,
            window, sinks, weights_16bit=True)
