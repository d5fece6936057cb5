"""Sampling where one token is likely and a great many equal ones are not: their weights' errors do not
cancel. Edges between tokens are then where the documentation says: off by at most vocab * 2^-43 +
2^-20 * (the share of weights below 2^-20 of the sum) of the sum."""
import numpy as np
import pytest

from tests.test_sample_gpu import sample, typed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab,below", [(100003, 14.0), (100003, 14.5), (100003, 15.0), (100003, 17.25), (1000003, 14.75),
                                         (1000003, 16.5)])
@pytest.mark.parametrize("rows", [8, 2000])
@pytest.mark.parametrize("top_p", [1.0, 0.99])
def test_many_equal_unlikely_tokens(cuda_lib, dtype, vocab, below, rows, top_p):
    rng = np.random.default_rng([vocab, int(100 * below), rows])
    if vocab > 500000:
        rows = min(rows, 700)
    x = np.full(vocab, -below)
    x[vocab // 3] = 0.0
    t = typed(x, dtype)
    # numbers over the whole row, next to edges (between two floats of the number, 2^-24 apart)
    w = np.exp(t.double().numpy())
    order = np.argsort(-t.double().numpy(), kind="stable")
    if top_p < 1:
        before = np.cumsum(w[order]) - w[order]
        w[order[before >= np.float64(np.float32(top_p)) * w.sum()]] = 0.0
    cdf = np.cumsum(w) / w.sum()
    pick = rng.integers(vocab, size=rows)
    u = np.where(np.arange(rows) % 2 == 0, rng.random(rows), cdf[pick] + rng.uniform(-1, 1, rows) * 2.0 ** -24)
    u = np.clip(u, 0, 1 - 2.0 ** -24).astype(np.float32)
    more = {"top_p": [top_p] * rows} if top_p < 1 else {}
    got = np.array(sample(cuda_lib, t.cuda().repeat(rows, 1), u, **more))
    small = w[(w > 0) & (w < 2.0 ** -20 * w.sum())].sum() / w.sum()
    off = vocab * 2.0 ** -43 + 2.0 ** -20 * small
    if top_p < 1:  # the border is off by as much, and one token more or less of those behind it is kept
        off = 3 * off + np.exp(t.double().numpy().min()) / w.sum()
    lo, hi = np.concatenate([[0.0], cdf])[got], cdf[got]
    assert (u >= lo - off).all() and (u <= hi + off).all(), f"off by {max((lo - u).max(), (u - hi).max()):.2e}, not {off:.2e}"
