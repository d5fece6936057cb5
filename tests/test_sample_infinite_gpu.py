"""Sampling from rows whose largest logit is infinite, or whose z = x / T passes the range of fp32: the
smaller logits have weights of 0 then, whichever the filter, the number and the CTAs of a row."""
import numpy as np
import pytest

from tests.test_sample_gpu import sample, typed

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = np.inf
MAX = float(np.finfo(np.float32).max)
# 110 numbers over [0, 1), closer together below 1
NUMBERS = np.concatenate([np.arange(100) / 100, [0.995, 0.999, 0.9995, 0.9999, 0.99999, 1e-3, 1e-6, 0.335, 0.667,
                                                 1 - 2.0 ** -24]]).astype(np.float32)
FILTERS = [{}, dict(top_k=2), dict(top_k=5), dict(top_k=2500), dict(top_p=0.3), dict(top_p=0.9), dict(top_p=0.999),
           dict(min_p=0.1), dict(top_k=2500, top_p=0.6, min_p=1e-6)]


def tokens_of(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The definition in 64 bits, for one row and many numbers."""
    top = x.max()
    order = np.argsort(-x, kind="stable")
    s = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(s == top, 1.0, np.exp((s - top) / temperature))
    keep = s > -INF
    if 0 < top_k < len(x):
        keep &= np.arange(len(x)) < top_k
    w = np.where(keep, w, 0.0)
    if top_p < 1:
        w = np.where(np.concatenate([[0.0], np.cumsum(w)[:-1]]) < top_p * w.sum(), w, 0.0)
    w = np.where(w >= min_p, w, 0.0)
    by_index = np.zeros(len(x))
    by_index[order] = w
    cdf = np.cumsum(by_index)
    return np.searchsorted(cdf, u.astype(np.float64) * cdf[-1], side="right").tolist()


def check(gdn, x, rows, dtype="float32", temperature=1.0, **settings):
    """`rows` times the same row, each with a number of its own."""
    t = typed(x, dtype)
    u = np.resize(NUMBERS, rows)
    logits = t.cuda().repeat(rows, 1)
    exact = t.double().numpy()
    for start in range(0, len(NUMBERS), rows):
        u = np.resize(np.roll(NUMBERS, -start), rows)
        got = sample(gdn, logits, u, temperature=[temperature] * rows, **{k: [v] * rows for k, v in settings.items()})
        exactly = {k: v if k == "top_k" else float(np.float32(v)) for k, v in settings.items()}
        want = tokens_of(exact, u, temperature=float(np.float32(temperature)), **exactly)
        assert got == want, f"{settings}, temperature {temperature}"


# rows of 8, 64, 150 and 330 at once: eight, four, two and one CTAs a row where the vocabulary is large
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("vocab,rows", [(3001, 110), (50257, 8), (50257, 64), (128000, 150), (50257, 330)])
@pytest.mark.parametrize("where", [[0], [-1], [1234], [7, 70, 2900], [0, 1, -2, -1]])
def test_infinite_logits(cuda_lib, dtype, vocab, rows, where):
    rng = np.random.default_rng([vocab, rows, len(where)])
    x = 2 * rng.standard_normal(vocab)
    x[where] = INF
    for settings in FILTERS:
        check(cuda_lib, x, rows, dtype, **settings)
    check(cuda_lib, x, rows, dtype, temperature=50.0, top_p=0.95)


@pytest.mark.parametrize("vocab,rows", [(3001, 110), (50257, 8), (50257, 330)])
@pytest.mark.parametrize("top", [MAX, -0.9 * MAX, 20.0, -20.0])
def test_products_past_the_range(cuda_lib, vocab, rows, top):
    """x log2(e) / T overflows: the largest float, or temperatures near the smallest."""
    rng = np.random.default_rng([vocab, rows])
    temperature = 1.0 if abs(top) > 1e30 else 8e-38
    x = top - np.abs(top) * (0.05 * rng.random(vocab) + 1e-3)
    x[[5, 2000, -3]] = top
    for settings in FILTERS:
        check(cuda_lib, x, rows, temperature=temperature, **settings)


def test_largest_floats_side_by_side(cuda_lib):
    """The largest float, its neighbour below and banned tokens at the lowest; an infinity beside them."""
    x = np.full(4099, -MAX)
    x[3], x[2500] = MAX, np.nextafter(np.float32(MAX), np.float32(0))
    for settings in FILTERS:
        check(cuda_lib, x, 110, **settings)
        check(cuda_lib, np.where(np.arange(4099) == 4000, INF, x), 110, **settings)
        check(cuda_lib, np.where(x > 0, -MAX, -INF), 110, **settings)
