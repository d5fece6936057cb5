"""The block over trees where a node's inputs are not finite: those who descend from it have NaN, nobody else
has anything of it, and neither has a commit along another branch."""
import numpy as np
import pytest

from tests.test_block_tree_gpu import Device, check_commit, close
from tests.tree_cases import Block, path_to, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s", [32, 64, 128, 256])
@pytest.mark.parametrize("n_nodes,kernel", [(7, 2), (24, 4), (64, 8)])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_inputs_of_one_branch(cuda_lib, s, n_nodes, kernel, value):
    rng = np.random.default_rng([s, n_nodes])
    trees = [random_tree(rng, n_nodes, chain=0.3) for _ in range(2)]
    c = Block(rng, trees, 2, 4, s, kernel)
    outs, after = zip(*(c.run(x) for x in range(c.n)))
    odd = [n_nodes // 2, n_nodes - 1]
    for x, i in enumerate(odd):
        c.qkv[x, i], c.z[x, i] = value, value
        c.alpha[x, i], c.b[x, i] = np.nan, np.nan
    d = Device(cuda_lib, c)
    got = d.tree()
    for x, tree in enumerate(trees):
        behind = [odd[x] in path_to(tree, i) for i in range(n_nodes)]
        close(got[x][~np.array(behind)], outs[x][~np.array(behind)], "the other branches")
        assert np.isnan(got[x][np.array(behind)]).any(-1).all()
    accepted = [max(i for i in range(n_nodes) if odd[x] not in path_to(trees[x], i)) + 1 for x in range(2)]
    check_commit(d, c, after, accepted)
    cuda_lib.gdn_device_error()
