"""Sampling at the hottest temperatures that a call takes, with logits as far apart as floats are."""
import numpy as np
import pytest

from tests.test_sample_gpu import sample
from tests.test_sample_infinite_gpu import FILTERS, MAX, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("temperature", [1e20, 1.2e30])
@pytest.mark.parametrize("vocab,rows", [(3001, 110), (50257, 8)])
def test_hottest(cuda_lib, temperature, vocab, rows):
    """Spread over all floats, in which the smaller logits have no weight, and over a few temperatures."""
    rng = np.random.default_rng(vocab)
    wide = rng.uniform(-1, 1, vocab) * MAX
    near = rng.standard_normal(vocab) * 3 * temperature
    for settings in FILTERS:
        check(cuda_lib, wide, rows, temperature=temperature, **settings)
        check(cuda_lib, near, rows, temperature=temperature, **settings)


def test_hotter_is_refused(cuda_lib):
    x = torch.tensor([[3e38, -3e38, 0.0]] * 4, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sample(cuda_lib, x, [0.5] * 4, err=err, temperature=[1e38, 2.0 ** 100, np.nextafter(np.float32(2.0 ** 100), np.float32(0)), 1.0])
    assert got[:2] == [-1, -1] and got[2:] == [0, 0] and err.item() == 2
