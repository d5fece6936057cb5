"""One dominant float16 key over a long, nearly flat tail: weights far below the row's largest,
which only count together, against the plain form in 64 bits.

The bound is the attention calls' (tests/attn_cases.py) and what float16 holds of a small
weight. Its steps end at 2^-24. Decode holds weights, in two parts, up to 2^14 and sums them
before rounding: a weight is off by at most 2^-25, 2^-39 of the largest. The prompt form holds
one part and a largest weight of 2^7 at least: 2^-32 of it. Over n keys a row's weights are
off by n times that, next to a sum of 1 or more."""
import numpy as np
import pytest

from tests.attn_cases import Cache, attention, bound
from tests.test_attn_decode_gpu import run as decode
from tests.test_attn_prefill_gpu import run as prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NATS = 17.5  # the tail's weights lie around 2^-25.2 of the largest


def strong_key(rng, n, hkv, d, at, dtype="float16"):
    """A sequence whose key `at` has the largest score by NATS, and value 0; the tail's values
    lie around 1."""
    c = Cache(torch, rng, [n], hkv, d, 64, dtype)
    k, v = np.zeros((n, hkv, d)), c.typed(1 + 0.25 * rng.standard_normal((n, hkv, d)))
    k[:, :, 1] = 0.1 * rng.standard_normal((n, hkv))
    k[at, :, 0], k[at, :, 1], v[at] = NATS, 0, 0
    c.k, c.v = [c.typed(k)], [v]
    row = c.table[c.slots[0]]
    for col in range(-(-n // c.ps)):
        part = slice(col * c.ps, min(n, (col + 1) * c.ps))
        m = part.stop - part.start
        c.k_pages[row[col], :, :m] = c.dev(c.k[0][part].transpose(1, 0, 2))
        c.v_pages[row[col], :, :m] = c.dev(v[part].transpose(1, 0, 2))
    return c


def ask(rows, hq, d):
    q = np.zeros((rows, hq, d))
    q[:, :, :2] = 1
    return q


def agree(got, ref, q, c, per_key):
    tol = bound(ref, q, c.k[0], c.v[0], 1.0, c.dtype, weights_16bit=per_key > 2.0 ** -39)
    tol += 2 * c.lens[0] * per_key * np.abs(c.v[0]).max()
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"off by {(err / tol).max():.2f} of the bound"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 20000])
@pytest.mark.parametrize("n_tokens", [1, 3])
def test_decode(cuda_lib, d, at, n_tokens):
    """More sequences (all over the same pages) than CTAs, so that a CTA holds long parts of a
    unit, the strong key's among them; and one sequence alone, split over all CTAs."""
    rng = np.random.default_rng([d, at])
    hkv = 2
    c = strong_key(rng, 32767, hkv, d, at)
    q = ask(n_tokens, hkv, d)
    ref = attention(q, c.k[0], c.v[0], c.lens[0] - n_tokens, 1.0, 0, 0)
    agree(decode(cuda_lib, c, q, n_tokens, hkv, scale=1.0).double().cpu().numpy(), ref, q, c, 2.0 ** -39)
    n = 160
    whole = Cache.__new__(Cache)
    whole.__dict__.update(c.__dict__)
    whole.lens, whole.pool = c.lens * n, n
    whole.d_table, whole.d_lens = c.d_table.repeat(n, 1), c.d_lens.repeat(n)
    out = decode(cuda_lib, whole, np.tile(q, (n, 1, 1)), n_tokens, hkv, scale=1.0, slots=False)
    for i, got in enumerate(out.double().cpu().numpy().reshape(n, n_tokens, hkv, d)):
        agree(got, ref, q, c, 2.0 ** -39)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 70000])
def test_prompt(cuda_lib, d, at):
    """A few new tokens after a long history: one row tile sees all of it."""
    rng = np.random.default_rng([d, at, 1])
    c = strong_key(rng, 131071, 1, d, at)
    q = ask(3, 2, d)
    ref = attention(q, c.k[0], c.v[0], c.lens[0] - 3, 1.0, 0, 0)
    agree(prefill(cuda_lib, c, q, [3], 2, scale=1.0).double().cpu().numpy(), ref, q, c, 2.0 ** -32)
