"""Forks from a pool that has run out of pages: only a fork that needs a page is refused."""
import numpy as np
import pytest

from tests.test_pages_gpu import Device, Model

pytestmark = pytest.mark.gpu


def exhausted(rng, ps, lens, max_pages=4):
    """Sequences of the given lengths in slots 0 .. and no page left; as many empty slots."""
    need = sum(-(-n // ps) for n in lens)
    m = Model(rng, 3 * len(lens), need, ps, max_pages)
    m.reserve(range(len(lens)), lens)
    assert not m.free() and m.errors == 0
    return m


@pytest.mark.parametrize("lens", [[13, 16, 0, 8], [16, 13, 24, 1, 0], [9, 9, 8]])
def test_full_pages_are_shared_without_a_free_one(cuda_lib, lens):
    """Parents with partly full last pages ahead of, between and behind parents that end on a
    page's edge, and an empty one."""
    m = exhausted(np.random.default_rng(len(lens)), 8, lens)
    d = Device(cuda_lib, m)
    parents, children = list(range(len(lens))), [len(lens) + i for i in range(len(lens))]
    for side in (m, d):
        side.fork(parents, children)
    d.same("fork without a free page")
    assert m.errors == sum(n % 8 > 0 for n in lens)
    assert all(m.lens[c] == (0 if n % 8 else n) for c, n in zip(children, lens))


def test_the_last_page_goes_to_the_first_that_asks(cuda_lib):
    m = exhausted(np.random.default_rng(1), 8, [16, 13, 12, 24, 8])
    m.truncate([4], [0])
    d = Device(cuda_lib, m)
    for side in (m, d):
        side.fork([0, 1, 2, 3, 0], [5, 6, 7, 8, 9])
    d.same("one free page")
    assert m.errors == 1 and m.lens[5:10].tolist() == [16, 13, 0, 24, 16]


def test_many_forks(cuda_lib):
    """More forks than the plan has threads, pages running out on the way."""
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.choice([0, 5, 8, 16, 21, 24], 1100)]
    m = exhausted(rng, 8, lens)
    m.truncate(range(0, 300, 7), [0] * len(range(0, 300, 7)))
    d = Device(cuda_lib, m)
    parents = [int(x) for x in rng.permutation(1100)]
    children = [1100 + i for i in range(1100)]
    for side in (m, d):
        side.fork(parents, children)
    d.same("many forks")
    assert 0 < m.errors < sum(n % 8 > 0 for n in lens)
