"""The block over trees of drafts and its commit, against the plain form in 64 bits and against the
block over chains."""
import numpy as np
import pytest

from tests.tree_cases import NO_NODE, Block, path_to, random_tree, valid

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Device:
    """A block's arrays on the device."""

    def __init__(self, gdn, c, err=None, slots="own"):
        self.gdn, self.c = gdn, c
        for name in ("qkv", "conv_w", "conv_state", "alpha", "b", "dt", "a", "z", "norm_w", "state"):
            setattr(self, name, dev(getattr(c, name).astype(np.float32)))
        self.parents = dev(np.array(c.trees, np.int32))
        self.out = torch.full((c.n, c.t, c.h, c.s), 7.0, device="cuda")
        sizes = (c.n, c.t, c.hk, c.h, c.s)
        self.tape = torch.full((gdn.gdn_block_tree_tape_size(*sizes),), 0xFF, device="cuda", dtype=torch.uint8)
        self.ws = torch.full((gdn.gdn_block_tree_workspace_size(*sizes),), 0xFF, device="cuda", dtype=torch.uint8)
        self.more = dict(slots=dev(np.array(c.slots if slots == "own" else slots, np.int32)), pool=c.pool, err_count=err)

    def tree(self, **more):
        c = self.c
        self.gdn.gdn_block_tree(self.qkv, self.conv_w, self.conv_state, self.alpha, self.b, self.dt, self.a,
                                self.z, self.norm_w, self.state, self.out, self.parents, c.n, c.t, c.hk, c.h,
                                c.s, c.kernel, c.scale, c.eps, c.eps, self.tape, self.ws, **self.more, **more)
        return self.out.cpu().numpy()

    def commit(self, accepted, **more):
        c = self.c
        self.gdn.gdn_block_tree_commit(self.qkv, self.conv_state, self.state, self.parents,
                                       dev(np.array(accepted, np.int32)), c.n, c.t, c.hk, c.h, c.s, c.kernel,
                                       self.tape, **self.more, **more)
        return self.state.cpu().numpy(), self.conv_state.cpu().numpy()


def close(got, ref, what):
    size = np.abs(ref).max() if ref.size else 0.0
    err = np.abs(got - ref)
    tol = 1e-4 + 1e-4 * max(size, 1.0)
    assert np.isfinite(got).all() and (err <= tol).all(), f"{what}: off by {err.max():.2e}, allowed {tol:.2e}"


def check_commit(d, c, after, accepted):
    before = d.state.cpu().numpy()
    state, conv = d.commit(accepted)
    for x, slot in enumerate(c.slots):
        if accepted[x] == 0:
            assert np.array_equal(state[slot], before[slot])
            continue
        want, hist = after[x][accepted[x] - 1]
        close(state[slot], want, f"state of sequence {x}")
        assert np.array_equal(conv[slot], hist.astype(np.float32)), f"history of sequence {x}"
    for slot in set(range(c.pool)) - set(c.slots):
        assert np.array_equal(state[slot], c.state[slot]) and np.array_equal(conv[slot], c.conv_state[slot])


@pytest.mark.parametrize("s", [32, 64, 128, 256])
@pytest.mark.parametrize("n_nodes,hk,h,kernel", [(1, 1, 1, 4), (2, 2, 4, 2), (9, 2, 6, 3), (17, 4, 4, 4), (33, 1, 3, 8), (64, 2, 2, 4)])
@pytest.mark.parametrize("chain", [0.0, 0.5, 1.0])
def test_trees(cuda_lib, s, n_nodes, hk, h, kernel, chain):
    rng = np.random.default_rng([s, n_nodes, int(10 * chain)])
    trees = [random_tree(rng, n_nodes, chain=chain),
             random_tree(rng, n_nodes, int(rng.integers(0, n_nodes + 1)), chain),
             random_tree(rng, n_nodes, chain=chain, roots=min(2, n_nodes))]
    c = Block(rng, trees, hk, h, s, kernel, pool=5, slots=[4, 0, 2])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = Device(cuda_lib, c, err)
    got = d.tree()
    after = []
    for x in range(c.n):
        out, states = c.run(x)
        after.append(states)
        close(got[x], out, f"sequence {x}")
        there, _ = valid(trees[x])
        assert (got[x][~np.array(there)] == 0).all()
    assert np.array_equal(d.state.cpu().numpy(), c.state) and np.array_equal(d.conv_state.cpu().numpy(), c.conv_state)
    # to the last node, to none where the tree is empty, to a node in the middle
    accepted = [n_nodes, sum(valid(trees[1])[0]), n_nodes // 2 + 1]
    check_commit(d, c, after, accepted)
    assert err.item() == 0


@pytest.mark.parametrize("decay", [0.01, 8.0])
def test_long_paths(cuda_lib, decay):
    """A chain of 64 whose decays hardly, or all but wholly, forget."""
    rng = np.random.default_rng(8)
    c = Block(rng, [list(range(-1, 63))] * 2, 2, 4, 128, 4, decay=decay)
    d = Device(cuda_lib, c)
    got = d.tree()
    runs = [c.run(x) for x in range(2)]
    for x in range(2):
        close(got[x], runs[x][0], f"sequence {x}")
    check_commit(d, c, [r[1] for r in runs], [64, 40])


@pytest.mark.parametrize("s", [64, 128])
def test_chain_is_the_prefill_block(cuda_lib, s):
    """A chain: the prefill block's outputs and states, up to rounding; the histories its bits."""
    rng = np.random.default_rng(9)
    n, t, hk, h, kernel = 3, 12, 2, 4, 4
    c = Block(rng, [list(range(-1, t - 1))] * n, hk, h, s, kernel)
    d = Device(cuda_lib, c)
    got = d.tree()
    state, conv, out = d.state.clone(), d.conv_state.clone(), torch.empty_like(d.out)
    ws = torch.empty(cuda_lib.gdn_block_prefill_workspace_size(n, t, hk, h, s), device="cuda", dtype=torch.uint8)
    cuda_lib.gdn_block_prefill(d.qkv, d.conv_w, conv, d.alpha, d.b, d.dt, d.a, d.z, d.norm_w, state, out, n, t,
                               hk, h, s, kernel, c.scale, c.eps, c.eps, ws)
    close(got, out.cpu().numpy(), "outputs")
    got_state, got_conv = d.commit([t] * n)
    close(got_state, state.cpu().numpy(), "states")
    assert np.array_equal(got_conv, conv.cpu().numpy())


def test_what_is_skipped_and_counted(cuda_lib):
    rng = np.random.default_rng(10)
    t = 6
    trees = [random_tree(rng, t) for _ in range(5)]
    trees[1][3] = 5
    trees[2][0] = -9
    c = Block(rng, trees, 2, 2, 64, 4, pool=6, slots=[0, 1, 2, 3, 4])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = Device(cuda_lib, c, err, slots=[0, 1, 2, 6, -1])
    got = d.tree()
    assert err.item() == 4  # two slots, two trees
    for x in range(3):
        close(got[x], c.run(x)[0], f"sequence {x}")
    assert (got[3:] == 7).all()
    err.zero_()
    state, conv = d.commit([t + 1, 4, 1, 1, 1])  # out of range; not there; its root is not there
    assert err.item() == 5
    assert np.array_equal(state, c.state) and np.array_equal(conv, c.conv_state)


def test_streams_and_replays(cuda_lib):
    """Both calls on a stream of their own and captured; replays see other trees and inputs."""
    rng = np.random.default_rng(11)
    n, t = 4, 10
    c = Block(rng, [random_tree(rng, t) for _ in range(n)], 2, 4, 128, 4)
    d = Device(cuda_lib, c)
    accepted = dev(np.array([t, 1, 5, 3], np.int32))

    def both(**more):
        cuda_lib.gdn_block_tree(d.qkv, d.conv_w, d.conv_state, d.alpha, d.b, d.dt, d.a, d.z, d.norm_w, d.state,
                                d.out, d.parents, n, t, 2, 4, 128, 4, c.scale, c.eps, c.eps, d.tape, d.ws, **more)
        cuda_lib.gdn_block_tree_commit(d.qkv, d.conv_state, d.state, d.parents, accepted, n, t, 2, 4, 128, 4,
                                       d.tape, **more)

    def check():
        torch.cuda.synchronize()
        for x, m in enumerate(accepted.tolist()):
            out, after = c.run(x)
            close(d.out[x].cpu().numpy(), out, f"sequence {x}")
            close(d.state[x].cpu().numpy(), after[m - 1][0], f"state {x}")

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(stream=side.cuda_stream)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(2):
        new = Block(rng, [random_tree(rng, t) for _ in range(n)], 2, 4, 128, 4)
        c.__dict__.update(new.__dict__)
        for name in ("qkv", "conv_w", "conv_state", "alpha", "b", "dt", "a", "z", "norm_w", "state"):
            getattr(d, name).copy_(dev(getattr(c, name).astype(np.float32)))
        d.parents.copy_(dev(np.array(c.trees, np.int32)))
        graph.replay()
        check()


def test_path_helper():
    assert path_to([-1, 0, 0, 2, NO_NODE], 3) == [0, 2, 3]
