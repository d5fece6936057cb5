"""Attention of trees of drafts over the paged cache, against the plain form in 64 bits."""
import numpy as np
import pytest

from tests import tree_cases
from tests.attn_cases import Cache, bound
from tests.test_attn_decode_gpu import run as decode
from tests.tree_cases import NO_NODE, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Call:
    """A call's tensors; `go` makes it once more."""

    def __init__(self, gdn, c, q, trees, hq, window=0, sinks=0, packed=False, err=None):
        self.gdn, self.c = gdn, c
        n, t = len(trees), len(trees[0])
        self.q = c.dev(q)
        if packed:
            wide = torch.full((q.shape[0], hq + 3, c.d), np.nan, dtype=c.k_pages.dtype, device="cuda")
            wide[:, :hq] = self.q
            self.q = wide[:, :hq]
        self.out = torch.full((n * t, hq, c.d), 7.0, dtype=c.k_pages.dtype, device="cuda")
        self.parents, self.err = ints(trees), err
        size = gdn.gdn_attn_tree_workspace_size(n, t, hq, c.hkv, c.d)
        self.ws = torch.randint(0, 256, (size,), device="cuda", dtype=torch.int32).to(torch.uint8)
        self.args = (n, t, hq, c.hkv, c.d, c.ps, c.n_pages, c.max_pages, window, sinks, c.d ** -0.5)

    def go(self, **more):
        c = self.c
        self.gdn.gdn_attn_tree(self.q, c.k_pages, c.v_pages, c.d_table, c.d_lens, self.out, self.parents,
                               *self.args, self.ws, slots=c.d_slots, pool=c.pool, err_count=self.err, **more)
        return self.out


def check(c, out, q, trees, window, sinks, skipped=()):
    """Every row against the 64-bit form; those of skipped sequences as they were."""
    t = len(trees[0])
    got = out.double().cpu().numpy().reshape(q.shape)
    for x, tree in enumerate(trees):
        mine = got[x * t:(x + 1) * t]
        if x in skipped:
            assert (mine == 7).all(), f"sequence {x} was not skipped"
            continue
        rows = q[x * t:(x + 1) * t]
        ref = tree_cases.attention(rows, c.k[x], c.v[x], tree, c.d ** -0.5, window, sinks)
        there, _ = tree_cases.valid(tree)
        there = np.array(there)
        assert (mine[~there] == 0).all(), f"sequence {x}: a node that is not there is not zero"
        if not there.any():
            continue
        assert np.isfinite(mine).all(), f"sequence {x}: values that are not finite"
        tol = bound(ref[there], rows[there], c.k[x], c.v[x], c.d ** -0.5, c.dtype, weights_16bit=True)
        err = np.abs(mine[there] - ref[there])
        assert (err <= tol).all(), f"sequence {x}: off by {(err / tol).max():.2f} of the bound"


def poison(c, q, trees):
    """What a node that is not there holds -- its query, its key and value -- is NaN."""
    t = len(trees[0])
    for x, tree in enumerate(trees):
        there, _ = tree_cases.valid(tree)
        for i in range(t):
            if not there[i] and c.lens[x] >= t:
                j = c.lens[x] - t + i
                page = int(c.table[c.slots[x], j // c.ps])
                c.k_pages[page, :, j % c.ps] = float("nan")
                c.v_pages[page, :, j % c.ps] = float("nan")
                q[x * t + i] = np.nan


def case(rng, lens, n_nodes, hkv, group, d, ps, dtype, ragged=False, **tree):
    c = Cache(torch, rng, lens, hkv, d, ps, dtype, pool=len(lens) + 2)
    trees = [random_tree(rng, n_nodes, int(rng.integers(0, n_nodes + 1)) if ragged else None, **tree) for _ in lens]
    q = c.queries(rng, [n_nodes] * len(lens), hkv * group)
    return c, trees, q


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_nodes,group", [(1, 1), (2, 3), (7, 2), (16, 4), (33, 5), (64, 2), (64, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2), (5, 0)])
def test_trees(cuda_lib, dtype, d, n_nodes, group, window, sinks):
    rng = np.random.default_rng([d, n_nodes, group, window])
    lens = [n_nodes, n_nodes + 1, 127 + n_nodes, 128 + n_nodes, 700]
    c, trees, q = case(rng, lens, n_nodes, 2, group, d, 16, dtype)
    out = Call(cuda_lib, c, q, trees, 2 * group, window, sinks).go()
    check(c, out, q, trees, window, sinks)
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("n_nodes,group,ps", [(9, 3, 8), (24, 4, 256), (64, 3, 32)])
@pytest.mark.parametrize("chain,roots", [(1.0, 1), (0.0, 1), (0.3, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 1), (200, 4)])
def test_padded_trees_and_forests(cuda_lib, dtype, n_nodes, group, ps, chain, roots, window, sinks):
    """Smaller trees padded, whole trees missing, several roots; what is not there holds NaN."""
    rng = np.random.default_rng([n_nodes, ps, roots, int(10 * chain)])
    lens = [n_nodes, 300, 65 + n_nodes, 1000, 64]
    c, trees, q = case(rng, lens, n_nodes, 3, group, 128, ps, dtype, ragged=True, chain=chain, roots=min(roots, n_nodes))
    trees[1] = [NO_NODE] * n_nodes
    trees[3] = random_tree(rng, n_nodes, n_nodes, chain, roots)
    clean_q = q.copy()
    poison(c, q, trees)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Call(cuda_lib, c, q, trees, 3 * group, window, sinks, packed=True, err=err).go()
    check(c, out, clean_q, trees, window, sinks)
    assert err.item() == 0
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("float16", 64), ("float32", 64), ("bfloat16", 256)])
@pytest.mark.parametrize("n_nodes,group", [(5, 2), (40, 4)])
def test_long_and_ragged(cuda_lib, dtype, d, n_nodes, group):
    """Units split over many CTAs beside many that are not."""
    rng = np.random.default_rng([d, n_nodes])
    lens = [20001, n_nodes] + [int(x) for x in rng.integers(n_nodes, 900, 40)]
    c, trees, q = case(rng, lens, n_nodes, 2, group, d, 64, dtype, ragged=True)
    out = Call(cuda_lib, c, q, trees, 2 * group).go()
    check(c, out, q, trees, 0, 0)
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype,group", [("bfloat16", 2), ("bfloat16", 6), ("float32", 2)])
def test_chain_is_the_decode_call(cuda_lib, dtype, group):
    rng = np.random.default_rng(3)
    lens = [7, 200, 3000]
    c = Cache(torch, rng, lens, 2, 128, 32, dtype)
    q = c.queries(rng, [7] * 3, 2 * group)
    out = Call(cuda_lib, c, q, [list(range(-1, 6))] * 3, 2 * group, 100, 3).go()
    c.check(out, q, [7] * 3, 128 ** -0.5, 100, 3, weights_16bit=True)
    want = decode(cuda_lib, c, q, 7, 2 * group, 100, 3)
    c.check(want, q, [7] * 3, 128 ** -0.5, 100, 3)


@pytest.mark.parametrize("dtype,n_nodes,group", [("bfloat16", 6, 2), ("bfloat16", 20, 4), ("float32", 6, 2)])
def test_what_is_skipped_and_counted(cuda_lib, dtype, n_nodes, group):
    """Slots and lengths out of range, caches shorter than the tree, parents that are not valid,
    pages out of range."""
    rng = np.random.default_rng(4)
    lens = [100, 90, 80, 70, 60, 50, 40]
    c, trees, q = case(rng, lens, n_nodes, 2, group, 64, 16, dtype)
    trees[3][2] = 2                      # its own parent
    trees[4] = [-1, 5] + trees[4][2:]    # a parent behind its node; what hangs from it goes too
    trees[5][0] = -7
    slots, kv_lens, table = c.slots.copy().astype(np.int32), c.kv_lens.copy(), c.table.copy()
    slots[0] = c.pool
    kv_lens[slots[1]] = n_nodes - 1
    kv_lens[slots[2]] = -3
    table[slots[6], 0] = c.n_pages       # hides 16 keys
    c.d_slots, c.d_lens, c.d_table = ints(slots), ints(kv_lens), ints(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Call(cuda_lib, c, q, trees, 2 * group, err=err).go()
    counted = err.item()
    assert counted >= 3 + 3 + 1
    c.k[6], c.v[6] = c.k[6][16:], c.v[6][16:]
    c.lens[6] -= 16
    check(c, out, q, trees, 0, 0, skipped=(0, 1, 2))
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype,n_nodes,group", [("bfloat16", 3, 4), ("float16", 30, 4), ("float32", 10, 4)])
def test_streams_and_replays(cuda_lib, dtype, n_nodes, group):
    """On another stream than the current one, two calls at once, and replayed with other trees."""
    rng = np.random.default_rng(5)
    lens = [900, n_nodes, 333]
    made = [case(rng, lens, n_nodes, 2, group, 128, 32, dtype, ragged=True) for _ in range(2)]
    calls = [Call(cuda_lib, c, q, trees, 2 * group) for c, trees, q in made]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for call, stream in zip(calls, side):
            call.go(stream=stream.cuda_stream)
    torch.cuda.synchronize()
    for call, (c, trees, q) in zip(calls, made):
        check(c, call.out, q, trees, 0, 0)
    c, trees, q = made[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls[0].go()
    for _ in range(3):
        trees = [random_tree(rng, n_nodes, int(rng.integers(1, n_nodes + 1))) for _ in lens]
        calls[0].parents.copy_(ints(trees))
        calls[0].out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check(c, calls[0].out, q, trees, 0, 0)
    first = calls[0].out.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, calls[0].out)  # the same bits every time
