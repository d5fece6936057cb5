"""Acceptance of trees of drafts: the walk and the cache rows it moves, against a plain walk."""
import numpy as np
import pytest

from tests.tree_cases import NO_NODE, path_to, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def walk(tree, tokens, sampled):
    """(path, next token)."""
    if tree[0] != -1:
        return [], -1
    path = [0]
    for i in range(1, len(tree)):
        if tree[i] == path[-1] and tokens[i] == sampled[path[-1]]:
            path.append(i)
    return path, sampled[path[-1]]


def plain_walk(tree, tokens, sampled):
    """The same, child by child from every node."""
    if tree[0] != -1:
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        child = [i for i in range(at + 1, len(tree)) if tree[i] == at and tokens[i] == sampled[at]]
        if not child:
            return path, sampled[at]
        path.append(child[0])


class Model:
    """Pools of slots with cached rows, trees behind them."""

    def __init__(self, gdn, rng, trees, lens, planes=3, hkv=2, ps=8, row=32, pool=None, vocab=4):
        self.gdn, self.n, self.t = gdn, len(trees), len(trees[0])
        self.planes, self.hkv, self.ps, self.row = planes, hkv, ps, row
        self.pool = pool or self.n
        self.slots = rng.permutation(self.pool)[:self.n].astype(np.int32)
        need = [-(-max(x, 1) // ps) for x in lens]
        self.n_pages, self.max_pages = sum(need) + 4, max(need) + 1
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.pool, self.max_pages), -1, np.int32)
        self.lens = np.zeros(self.pool, np.int32)
        at = 0
        for s, m, x in zip(self.slots, need, lens):
            self.table[s, :m] = ids[at:at + m]
            self.lens[s] = x
            at += m
        self.pages = rng.integers(0, 256, (planes, self.n_pages, hkv, ps, row)).astype(np.uint8)
        self.trees = np.array(trees, np.int32)
        self.tokens = rng.integers(0, vocab, self.trees.shape).astype(np.int32)
        self.sampled = rng.integers(0, vocab, self.trees.shape).astype(np.int32)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go(self, with_pages=True, **more):
        n, t = self.n, self.t
        outs = [torch.full((n,), 77, dtype=torch.int32, device="cuda") for _ in range(4)]
        path = torch.full((n, t), 77, dtype=torch.int32, device="cuda")
        pages = torch.from_numpy(self.pages).cuda()
        cache = (pages, ints(self.table), ints(self.lens), self.hkv, self.ps, self.planes, self.n_pages,
                 self.hkv * self.ps * self.row, self.max_pages) if with_pages else ()
        if not with_pages:
            outs[2] = None
        self.gdn.gdn_tree_accept(ints(self.trees), ints(self.tokens), ints(self.sampled), outs[0], outs[1], outs[2],
                                 outs[3], path, n, t, *cache, slots=ints(self.slots), pool=self.pool,
                                 err_count=self.err, **more)
        torch.cuda.synchronize()
        return [None if x is None else x.tolist() for x in outs], path.cpu().numpy(), pages.cpu().numpy()

    def want(self, skipped=()):
        pages, outs, paths = self.pages.copy(), [[], [], [], []], np.full((self.n, self.t), -1)
        for x in range(self.n):
            slot = self.slots[x]
            path, token = ([], -1) if x in skipped else plain_walk(self.trees[x].tolist(), self.tokens[x], self.sampled[x])
            length = int(self.lens[slot]) if 0 <= slot < self.pool else 0
            base = length - self.t
            outs[0].append(path[-1] + 1 if path else 0)
            outs[1].append(len(path))
            outs[2].append(max(length, 0) if x in skipped else base + len(path))
            outs[3].append(int(token))
            paths[x, :len(path)] = path
            for i, node in enumerate(path):
                (sp, sr), (dp, dr) = divmod(base + node, self.ps), divmod(base + i, self.ps)
                pages[:, self.table[slot, dp], :, dr] = pages[:, self.table[slot, sp], :, sr]
        return outs, paths, pages


def test_the_two_walks_agree():
    rng = np.random.default_rng(0)
    for _ in range(200):
        tree = random_tree(rng, 12)
        tokens, sampled = rng.integers(0, 3, 12), rng.integers(0, 3, 12)
        assert walk(tree, tokens, sampled) == plain_walk(tree, tokens, sampled)


@pytest.mark.parametrize("n_nodes", [1, 2, 5, 16, 31, 32, 33, 64])
@pytest.mark.parametrize("vocab,chain", [(1, 0.3), (2, 0.5), (4, 0.0), (1, 1.0)])
@pytest.mark.parametrize("planes,hkv,ps,row", [(1, 1, 8, 16), (4, 3, 16, 128), (2, 5, 64, 48)])
def test_walks_and_moves(cuda_lib, n_nodes, vocab, chain, planes, hkv, ps, row):
    """Vocabularies so small that paths are long and children alike; rows that cross pages."""
    rng = np.random.default_rng([n_nodes, vocab, planes])
    trees = [random_tree(rng, n_nodes, int(rng.integers(0, n_nodes + 1)) if x % 2 else None, chain) for x in range(9)]
    lens = [n_nodes + int(rng.integers(0, 40)) for _ in trees]
    m = Model(cuda_lib, rng, trees, lens, planes, hkv, ps, row, pool=13, vocab=vocab)
    outs, path, pages = m.go()
    want, want_path, want_pages = m.want()
    assert outs == want
    assert np.array_equal(path, want_path)
    assert np.array_equal(pages, want_pages)
    assert m.err.item() == 0
    outs, path, _ = m.go(with_pages=False)
    assert outs[:2] + outs[3:] == want[:2] + want[3:] and np.array_equal(path, want_path)


def test_what_is_skipped_and_counted(cuda_lib):
    rng = np.random.default_rng(1)
    t = 10
    trees = [random_tree(rng, t) for _ in range(7)]
    trees[4][2] = 7                            # not valid, and nobody's child on the path
    trees[5][0] = NO_NODE                      # nothing is kept
    trees[5][1:] = [NO_NODE] * (t - 1)
    m = Model(cuda_lib, rng, trees, [30] * 7, vocab=1)
    m.lens[m.slots[1]] = t - 1
    m.lens[m.slots[2]] = -1
    m.lens[m.slots[3]] = m.max_pages * m.ps + 1
    m.slots[0] = 99
    outs, path, pages = m.go()
    want, want_path, want_pages = m.want(skipped=(0, 1, 2, 3))
    assert outs == want and np.array_equal(path, want_path) and np.array_equal(pages, want_pages)
    assert m.err.item() == 5


def test_pages_out_of_range_do_not_move(cuda_lib):
    rng = np.random.default_rng(2)
    t = 8
    tree = [-1, 0, 0, 2, 3, 4, 5, 6]
    m = Model(cuda_lib, rng, [tree, tree], [16, 16], ps=8, vocab=1)
    m.tokens[:, 1] = 5                          # the path is 0, 2, 3, ... 7
    good = m.table[m.slots[1]].copy()
    m.table[m.slots[1], 1] = m.n_pages          # holds all rows of the tree
    outs, path, pages = m.go()
    assert outs[1] == [7, 7] and m.err.item() == 6
    want = m.pages.copy()
    base = 8
    for i, node in enumerate([0, 2, 3, 4, 5, 6, 7]):
        row = lambda j: (m.table[m.slots[0], j // 8], j % 8)  # noqa: E731
        (sp, sr), (dp, dr) = row(base + node), row(base + i)
        want[:, dp, :, dr] = m.pages[:, sp, :, sr]
    assert np.array_equal(pages, want)
    assert good[1] != m.table[m.slots[1], 1]
    assert path_to(tree, 7) == [0, 2, 3, 4, 5, 6, 7]


def test_captured_and_replayed(cuda_lib):
    rng = np.random.default_rng(3)
    n, t = 5, 20
    parents, tokens, sampled = (torch.zeros(n, t, dtype=torch.int32, device="cuda") for _ in range(3))
    outs = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3)]
    path = torch.zeros(n, t, dtype=torch.int32, device="cuda")

    def call():
        cuda_lib.gdn_tree_accept(parents, tokens, sampled, outs[0], outs[1], None, outs[2], path, n, t)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        trees = [random_tree(rng, t) for _ in range(n)]
        a, b = rng.integers(0, 2, (n, t)), rng.integers(0, 2, (n, t))
        for x, y in ((parents, trees), (tokens, a), (sampled, b)):
            x.copy_(ints(y))
        graph.replay()
        torch.cuda.synchronize()
        for x in range(n):
            want, token = plain_walk(trees[x], a[x], b[x])
            assert path[x, :len(want)].tolist() == want and outs[2][x].item() == token
            assert outs[0][x].item() == want[-1] + 1 and outs[1][x].item() == len(want)
