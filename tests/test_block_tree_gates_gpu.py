"""The block over trees where gates forget everything at some nodes: decays far below fp32's range, alpha at
infinity, beta 0 and 1. What lies behind such a node starts from nothing, as it does in a chain."""
import numpy as np
import pytest

from tests.test_block_tree_gpu import Device, check_commit, close
from tests.tree_cases import Block, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s", [32, 64, 128, 256])
@pytest.mark.parametrize("strength", [90.0, 300.0, 1e5, 1e9, 1e13, 1e20, 1e38, np.inf])
@pytest.mark.parametrize("n_nodes,chain", [(17, 1.0), (48, 0.6)])
def test_nodes_that_forget(cuda_lib, s, strength, n_nodes, chain):
    rng = np.random.default_rng([s, n_nodes])
    c = Block(rng, [random_tree(rng, n_nodes, chain=chain) for _ in range(2)], 2, 4, s, 4)
    forget = rng.random((2, n_nodes)) < 0.2
    forget[:, 0] = True
    c.alpha[forget] = strength           # softplus of it, times a of some -1
    c.b[rng.random(c.b.shape) < 0.1] = np.inf
    c.b[rng.random(c.b.shape) < 0.1] = -np.inf
    with np.errstate(over="ignore"):
        outs, after = zip(*(c.run(x) for x in range(c.n)))
    d = Device(cuda_lib, c)
    close(d.tree(), np.array(outs), "the block")
    check_commit(d, c, after, [n_nodes, n_nodes // 2])
    cuda_lib.gdn_device_error()
