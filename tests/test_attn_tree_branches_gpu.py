"""Keys and values that are not finite at a node, or at a key that only some nodes' windows reach: the nodes
that see it have what the formula gives there, all others are as if it were not."""
import numpy as np
import pytest

from tests import tree_cases
from tests.attn_cases import bound
from tests.test_attn_tree_gpu import Call, case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIZES = [(2, 2), (4, 2), (7, 2), (9, 3), (16, 4), (33, 5), (64, 2), (64, 8)]


def put(c, x, j, k=None, v=None, head=None, dim=None):
    """Other values at position j of sequence x: the whole row, or one element of one head."""
    page, at = int(c.table[c.slots[x], j // c.ps]), j % c.ps
    for value, plane, rows in ((k, c.k_pages, c.k), (v, c.v_pages, c.v)):
        if value is None:
            continue
        heads = slice(None) if head is None else head
        dims = slice(None) if dim is None else dim
        plane[page, heads, at, dims] = value
        rows[x][j, heads, dims] = value


def without_zero_weights(q, k, v, tree, scale, window, sinks):
    """As tree_cases.attention, keys with scores of -infinity left out."""
    v = v.copy()
    out = np.zeros(q.shape)
    for i in range(len(tree)):
        for h in range(q.shape[1]):
            kv = h // (q.shape[1] // k.shape[1])
            s = scale * (k[:, kv] @ q[i, h])
            out[i, h] = tree_cases.attention(q[i:i + 1, h:h + 1].repeat(len(tree), 0), k[:, kv:kv + 1],
                                             np.where((s == -np.inf)[:, None, None], 0.0, v[:, kv:kv + 1]),
                                             tree, scale, window, sinks)[i, 0]
    return out


def check(c, out, q, trees, window, sinks, two_parts=False):
    """Where a score is -infinity and its value is not finite the formula has 0 times an infinity, which is no
    number: there the output may be NaN, or what it is without that key (a part of a split row that has
    no weight at all is left out as a whole). two_parts: the weights may be held in two parts of 16 bits, hi + lo,
    of which lo is 0 or negative as often as not, and hi * infinity + lo * infinity is NaN then."""
    n = len(trees[0])
    got = out.double().cpu().numpy().reshape(q.shape)
    for x, tree in enumerate(trees):
        mine, rows = got[x * n:(x + 1) * n], q[x * n:(x + 1) * n]
        with np.errstate(invalid="ignore", over="ignore"):
            ref = tree_cases.attention(rows, c.k[x], c.v[x], tree, c.d ** -0.5, window, sinks)
        k, v = (np.where(np.isfinite(y[x]), y[x], 0.0) for y in (c.k, c.v))
        finite = np.isfinite(ref)
        tol = bound(np.where(finite, ref, 0.0), rows, k, v, c.d ** -0.5, c.dtype, weights_16bit=True)
        with np.errstate(invalid="ignore"):
            assert (np.abs(mine - ref)[finite] <= tol[finite]).all(), f"sequence {x}: nodes that do not see it are off"
        if two_parts:
            mine = np.where(np.isinf(ref) & np.isnan(mine), ref, mine)
        other = np.isnan(mine) != np.isnan(ref)
        if other.any():
            with np.errstate(invalid="ignore", over="ignore"):
                less = without_zero_weights(rows, c.k[x], c.v[x], tree, c.d ** -0.5, window, sinks)
            assert not np.isnan(mine[other]).any(), f"sequence {x}: NaN elsewhere"
            tol = bound(np.where(np.isfinite(less), less, 0.0), rows, k, v, c.d ** -0.5, c.dtype, weights_16bit=True)
            assert (np.abs(mine - less)[other] <= tol[other]).all(), f"sequence {x}: neither NaN nor without the key"
        inf = np.isinf(ref)
        assert np.array_equal(mine[inf], ref[inf]), f"sequence {x}: infinities"


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_nodes,group", SIZES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_values_of_one_branch(cuda_lib, dtype, d, n_nodes, group, window, sinks):
    rng = np.random.default_rng([d, n_nodes, group, window])
    lens = [n_nodes, 127 + n_nodes, 128 + n_nodes, 700, 5003]
    c, trees, q = case(rng, lens, n_nodes, 2, group, d, 16, dtype, chain=0.3)
    for x, value in enumerate([np.inf, -np.inf, np.nan, np.inf, -np.inf]):
        base = lens[x] - n_nodes
        put(c, x, base + n_nodes - 1, v=value)                       # a whole row, of the last node
        put(c, x, base + n_nodes // 2, v=np.nan, head=1, dim=d - 3)  # an element of an inner one
        put(c, x, base + n_nodes // 3, v=np.inf, head=0, dim=5)
        if window and base > window:  # the oldest key that a root still sees
            put(c, x, base - window + 1, v=value, head=0, dim=17)
    out = Call(cuda_lib, c, q, trees, 2 * group, window, sinks).go()
    check(c, out, q, trees, window, sinks, two_parts=dtype != "float32")
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_nodes,group", SIZES)
def test_keys_of_one_branch(cuda_lib, dtype, d, n_nodes, group):
    rng = np.random.default_rng([d, n_nodes, group])
    lens = [n_nodes, 127 + n_nodes, 700]
    c, trees, q = case(rng, lens, n_nodes, 2, group, d, 16, dtype, chain=0.3)
    for x, value in enumerate([np.inf, -np.inf, np.nan]):
        base = lens[x] - n_nodes
        put(c, x, base + n_nodes - 1, k=value, head=1, dim=3)
        put(c, x, base + n_nodes // 2, k=-value, v=value, head=0, dim=d - 1)
    out = Call(cuda_lib, c, q, trees, 2 * group).go()
    check(c, out, q, trees, 0, 0, two_parts=dtype != "float32")
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_nodes,group", [(4, 2), (9, 3), (33, 5)])
def test_values_that_all_see(cuda_lib, dtype, d, n_nodes, group):
    """In front of the tree: every node has the infinity (whichever form its rows take), or NaN."""
    rng = np.random.default_rng([d, n_nodes])
    lens = [500, 900, 333]
    c, trees, q = case(rng, lens, n_nodes, 2, group, d, 16, dtype)
    for x, value in enumerate([np.inf, -np.inf, np.nan]):
        put(c, x, 37, v=value, head=0, dim=11)
        put(c, x, 200, v=value, head=1, dim=0)
    out = Call(cuda_lib, c, q, trees, 2 * group).go()
    check(c, out, q, trees, 0, 0, two_parts=dtype != "float32")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_nodes,group", [(3, 1), (4, 2), (9, 3)])
def test_largest_floats(cuda_lib, d, n_nodes, group):
    """fp32 values above bf16's largest, at a key that has nearly all of the weight."""
    rng = np.random.default_rng([d, n_nodes])
    c, trees, q = case(rng, [300], n_nodes, 2, group, d, 16, "float32")
    top = float(np.finfo(np.float32).max)
    q = c.typed(np.abs(q))
    c.k[0][50] = c.typed(np.full((2, d), 40.0))
    c.k_pages[int(c.table[c.slots[0], 50 // 16]), :, 50 % 16] = 40.0
    put(c, 0, 50, v=top, head=0, dim=7)
    put(c, 0, 50, v=-top, head=1, dim=d - 2)
    got = Call(cuda_lib, c, q, trees, 2 * group).go().double().cpu().numpy().reshape(q.shape)
    ref = tree_cases.attention(q, c.k[0], c.v[0], trees[0], d ** -0.5, 0, 0)
    assert np.isfinite(got).all()
    tol = bound(ref, q, c.k[0], c.v[0], d ** -0.5, "float32")
    assert (np.abs(got - ref)[..., [7, d - 2]] <= tol[..., [7, d - 2]]).all()
