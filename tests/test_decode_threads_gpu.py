"""The block's decode called from several host threads at once, each with heads and batches of its own."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Decode:
    def __init__(self, gdn, rng, n, hk, h, s):
        f = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()  # noqa: E731
        self.gdn, self.sizes, c = gdn, (n, hk, h, s, 4), (2 * hk + h) * s
        self.ins = [f(n, c), f(c, 4), f(n, c, 3), f(n, h), f(n, h), f(h), -f(h).abs(), f(n, h, s), f(s), 0.1 * f(n, h, s, s)]
        self.out = torch.zeros(n, h, s, device="cuda")

    def start(self):
        """The arrays of a run, its histories and states as they were."""
        return [x.clone() for x in self.ins] + [torch.zeros_like(self.out)]

    def step(self, arrays, stream=None):
        self.gdn.gdn_block_decode(*arrays, *self.sizes, self.sizes[3] ** -0.5, 1e-6, 1e-6, stream=stream)


# (state size, (sequences, k-heads, v-heads) of the threads): a head's rows in parts, whose number hangs on the
# batch, and the persistent form with stages as its heads leave room for
@pytest.mark.parametrize("s,sizes", [(256, [(2, 1, 4), (2, 1, 2), (1, 1, 4), (3, 1, 2)]),
                                     (128, [(160, 2, 2), (160, 2, 16), (160, 2, 4), (2, 1, 8)]),
                                     (64, [(160, 2, 2), (160, 2, 16), (2, 1, 8), (160, 2, 6)]), (32, [(2, 1, 8), (300, 2, 4)])])
def test_sizes_at_once(cuda_lib, s, sizes):
    """The same bits as one thread's steps."""
    rng = np.random.default_rng(s)
    decodes = [Decode(cuda_lib, rng, *x, s) for x in sizes]
    steps, wanted = 1000, []
    for d in decodes:
        arrays = d.start()
        for _ in range(steps):
            d.step(arrays)
        wanted.append(arrays)
    runs = [d.start() for d in decodes]
    torch.cuda.synchronize()
    failed = []

    def go(d, arrays):
        stream = torch.cuda.Stream()
        try:
            for _ in range(steps):
                d.step(arrays, stream=stream.cuda_stream)
        except Exception as e:  # noqa: BLE001 (looked at below)
            failed.append(e)

    threads = [threading.Thread(target=go, args=x) for x in zip(decodes, runs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for arrays, want in zip(runs, wanted):
        assert all(torch.equal(a, b) for a, b in zip(arrays, want))
