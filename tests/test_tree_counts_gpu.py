"""What err_count holds behind the tree calls: a sequence once, however many units, heads and CTAs look at it."""
import numpy as np
import pytest

from tests.test_attn_tree_gpu import Call, case, check, ints
from tests.test_block_tree_gpu import Device
from tests.tree_cases import Block, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,n_nodes,hkv,group", [("bfloat16", 64, 6, 4, 2), ("bfloat16", 128, 20, 4, 4), ("float16", 128, 64, 3, 6),
                                                       ("bfloat16", 256, 24, 2, 8), ("float32", 64, 9, 4, 3), ("float32", 256, 64, 2, 2),
                                                       ("float16", 64, 3, 1, 40)])
def test_attention(cuda_lib, dtype, d, n_nodes, hkv, group):
    rng = np.random.default_rng([d, n_nodes])
    lens = [100, 9000, 8000, 7000, 6000, 5000, 4000]
    c, trees, q = case(rng, lens, n_nodes, hkv, group, d, 64, dtype)
    trees[3][2] = 2                      # its own parent
    trees[4] = [-1, 5] + trees[4][2:]    # a parent behind its node
    trees[5][0] = -7                     # no such value, and nothing else of the tree is there
    slots, kv_lens = c.slots.copy().astype(np.int32), c.kv_lens.copy()
    slots[0] = c.pool
    kv_lens[slots[1]] = n_nodes - 1
    kv_lens[slots[2]] = -3
    c.d_slots, c.d_lens = ints(slots), ints(kv_lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = Call(cuda_lib, c, q, trees, hkv * group, err=err)
    out = call.go()
    assert err.item() == 6
    call.go()
    assert err.item() == 12
    if d == 64:
        check(c, out, q, trees, 0, 0, skipped=(0, 1, 2))


@pytest.mark.parametrize("s", [32, 64, 128, 256])
def test_block_and_commit(cuda_lib, s):
    rng = np.random.default_rng(s)
    trees = [random_tree(rng, 33) for _ in range(5)]
    trees[1][4] = 4
    trees[2][0] = 7
    c = Block(rng, trees, 2, 8, s, 4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = Device(cuda_lib, c, err, slots=[0, 1, 2, -1, 5])
    d.tree()
    assert err.item() == 4
    err.zero_()
    d.commit([34, 5, 0, 1, 1])  # behind the tree, a node that is not there, nothing, two slots out of range
    assert err.item() == 4
