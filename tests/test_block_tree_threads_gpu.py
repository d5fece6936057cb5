"""The block over trees called from several host threads at once, each with trees of its own size."""
import threading

import numpy as np
import pytest

from tests.test_block_tree_gpu import Device, close
from tests.tree_cases import Block, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s", [32, 64, 128, 256])
def test_two_sizes_at_once(cuda_lib, s):
    rng = np.random.default_rng(s)
    cases = [Block(rng, [random_tree(rng, n) for _ in range(2)], 1, 2, s, 4) for n in (1, 64, 7, 40)]
    wanted = [np.array([c.run(x)[0] for x in range(c.n)]) for c in cases]
    devs = [Device(cuda_lib, c) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def go(d):
        c, stream = d.c, torch.cuda.Stream()
        try:
            for _ in range(1500):
                cuda_lib.gdn_block_tree(d.qkv, d.conv_w, d.conv_state, d.alpha, d.b, d.dt, d.a, d.z, d.norm_w, d.state,
                                        d.out, d.parents, c.n, c.t, c.hk, c.h, c.s, c.kernel, c.scale, c.eps, c.eps,
                                        d.tape, d.ws, stream=stream.cuda_stream, **d.more)
        except Exception as e:  # noqa: BLE001 (looked at below)
            failed.append(e)

    threads = [threading.Thread(target=go, args=(d,)) for d in devs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for d, want in zip(devs, wanted):
        close(d.out.cpu().numpy(), want, f"trees of {d.c.t}")


@pytest.mark.parametrize("s", [64, 128])
def test_captured_large_then_called_small(cuda_lib, s):
    """A captured call of large trees is replayed behind a call of small ones."""
    rng = np.random.default_rng(s)
    large, small = (Device(cuda_lib, Block(rng, [random_tree(rng, n)], 1, 2, s, 4)) for n in (64, 2))
    want = large.c.run(0)[0][None]
    large.tree()
    graph = torch.cuda.CUDAGraph()
    c, d = large.c, large
    with torch.cuda.graph(graph):
        cuda_lib.gdn_block_tree(d.qkv, d.conv_w, d.conv_state, d.alpha, d.b, d.dt, d.a, d.z, d.norm_w, d.state, d.out,
                                d.parents, c.n, c.t, c.hk, c.h, c.s, c.kernel, c.scale, c.eps, c.eps, d.tape, d.ws, **d.more)
    small.tree()
    d.out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    close(d.out.cpu().numpy(), want, "replayed")
