"""A call as the first thing that a host thread does with the GPU."""
import threading

import numpy as np
import pytest

from tests.attn_cases import Cache
from tests.test_attn_tree_gpu import Call, check
from tests.test_block_tree_gpu import Device, close
from tests.tree_cases import Block, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def in_new_thread(call):
    failed = []

    def go():
        try:
            call()
        except Exception as e:  # noqa: BLE001 (looked at below)
            failed.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed


@pytest.mark.parametrize("stream", [None, "side"])
def test_attention(cuda_lib, stream):
    rng = np.random.default_rng(1)
    stream = None if stream is None else torch.cuda.Stream().cuda_stream
    lens = [40, 333]
    for n_nodes in (3, 30):
        c = Cache(torch, rng, lens, 2, 64, 16, "bfloat16")
        trees = [random_tree(rng, n_nodes) for _ in lens]
        q = c.queries(rng, [n_nodes] * 2, 4)
        call = Call(cuda_lib, c, q, trees, 4)
        in_new_thread(lambda: call.go(stream=stream))
        check(c, call.out, q, trees, 0, 0)
    m, d = 4, 64
    c = Cache(torch, rng, lens, 2, d, 16, "float16")
    q = c.queries(rng, [m] * 2, 4)
    qd = c.dev(q)
    cu = torch.tensor([0, m, 2 * m], dtype=torch.int32, device="cuda")
    shared = (2, d, c.ps, c.n_pages, c.max_pages, 0, 0, d ** -0.5)
    more = dict(slots=c.d_slots, pool=c.pool, stream=stream)
    out = torch.full((2 * m, 4, d), 7.0, dtype=qd.dtype, device="cuda")
    ws = torch.zeros(cuda_lib.gdn_attn_decode_workspace_size(2, m, 4, 2, d), dtype=torch.uint8, device="cuda")
    in_new_thread(lambda: cuda_lib.gdn_attn_decode(qd, c.k_pages, c.v_pages, c.d_table, c.d_lens, out, 2, m, 4, *shared,
                                                   ws, **more))
    c.check(out, q, [m] * 2, d ** -0.5, 0, 0)
    out = torch.full((2 * m, 4, d), 7.0, dtype=qd.dtype, device="cuda")
    ws = torch.zeros(max(16, cuda_lib.gdn_attn_prefill_workspace_size(2, 2 * m, 4, 2, d)), dtype=torch.uint8, device="cuda")
    in_new_thread(lambda: cuda_lib.gdn_attn_prefill(qd, c.k_pages, c.v_pages, c.d_table, c.d_lens, out, cu, 2, 2 * m, m, 4,
                                                    *shared, ws, **more))
    c.check(out, q, [m] * 2, d ** -0.5, 0, 0, weights_16bit=True)


@pytest.mark.parametrize("s", [32, 64, 128, 256])
def test_block(cuda_lib, s):
    rng = np.random.default_rng(s)
    c = Block(rng, [random_tree(rng, 9) for _ in range(2)], 1, 2, s, 4)
    d = Device(cuda_lib, c)
    in_new_thread(lambda: cuda_lib.gdn_block_tree(
        d.qkv, d.conv_w, d.conv_state, d.alpha, d.b, d.dt, d.a, d.z, d.norm_w, d.state, d.out, d.parents, c.n, c.t, c.hk,
        c.h, c.s, c.kernel, c.scale, c.eps, c.eps, d.tape, d.ws, **d.more))
    close(d.out.cpu().numpy(), np.array([c.run(x)[0] for x in range(c.n)]), "the block")
