"""Trees of drafts where a call's data and its work lie elsewhere: cache pages past 2^32 bytes, state
pools past 2^31 rows' bytes, scales that are not positive, infinities where nobody looks, workspaces that
two captured graphs share, and no call allocating."""
import numpy as np
import pytest

from tests import tree_cases
from tests.attn_cases import bound
from tests.test_attn_places_gpu import move_up
from tests.test_attn_tree_gpu import Call, case, check, ints
from tests.test_block_tree_gpu import Device, close
from tests.test_sample_gpu import define, sample
from tests.test_tree_accept_gpu import Model
from tests.tree_cases import Block, random_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def plain(c):
    """Outputs [n][t][h][s] of a block's case, and what lies behind every node of its sequences."""
    outs, after = zip(*(c.run(x) for x in range(c.n)))
    return np.array(outs), after


@pytest.mark.parametrize("dtype,d,ps,n_nodes,group", [("bfloat16", 128, 256, 20, 4), ("float16", 64, 16, 64, 3),
                                                      ("float32", 128, 64, 12, 2), ("bfloat16", 256, 32, 3, 2)])
def test_pages_past_32_bits(cuda_lib, dtype, d, ps, n_nodes, group):
    rng = np.random.default_rng([d, ps])
    c, trees, q = case(rng, [300, n_nodes + 13], n_nodes, 2, group, d, ps, dtype)
    move_up(c, 1 << 32)
    check(c, Call(cuda_lib, c, q, trees, 2 * group).go(), q, trees, 0, 0)
    cuda_lib.gdn_device_error()


def test_accepted_rows_past_32_bits(cuda_lib):
    """Planes of more than 2^32 bytes, the sequences' pages at their ends."""
    rng = np.random.default_rng(1)
    trees = [random_tree(rng, 9) for _ in range(3)]
    m = Model(cuda_lib, rng, trees, [40, 9, 33], planes=2, vocab=2)
    want = m.want()
    page_bytes = m.hkv * m.ps * m.row
    first = (1 << 32) // page_bytes + 1
    big = torch.empty(2, first + m.n_pages, *m.pages.shape[2:], dtype=torch.uint8, device="cuda")
    big[:, first:] = torch.from_numpy(m.pages).cuda()
    outs = [torch.full((3,), 77, dtype=torch.int32, device="cuda") for _ in range(4)]
    path = torch.full((3, 9), 77, dtype=torch.int32, device="cuda")
    table = np.where(m.table >= 0, m.table + first, -1)
    cuda_lib.gdn_tree_accept(ints(trees), ints(m.tokens), ints(m.sampled), outs[0], outs[1], outs[2], outs[3], path,
                             3, 9, big, ints(table), ints(m.lens), m.hkv, m.ps, 2, first + m.n_pages, page_bytes,
                             m.max_pages, slots=ints(m.slots), pool=m.pool)
    assert [x.tolist() for x in outs] == want[0]
    assert np.array_equal(path.cpu().numpy(), want[1])
    assert np.array_equal(big[:, first:].cpu().numpy(), want[2])


@pytest.mark.parametrize("s,h,first", [(128, 32, 2100), (64, 32, 8400)])
def test_state_pools_past_32_bits(cuda_lib, s, h, first):
    """State rows that lie past 2^32 bytes of their pool (slots' places are counted in 64 bits)."""
    rng = np.random.default_rng(s)
    c = Block(rng, [random_tree(rng, 6) for _ in range(2)], h // 2, h, s, 4, pool=2)
    d = Device(cuda_lib, c)
    pool = first + 2
    state = torch.empty(pool, *d.state.shape[1:], device="cuda")
    conv = torch.empty(pool, *d.conv_state.shape[1:], device="cuda")
    assert state.numel() * 4 > 1 << 32
    state[first:], conv[first:] = d.state, d.conv_state
    d.state, d.conv_state = state, conv
    d.more = dict(slots=ints(np.array(c.slots) + first), pool=pool)
    ref, after = plain(c)
    close(d.tree(), ref, "the block")
    accepted = [3, 6]
    d.commit(accepted)
    for x, slot in enumerate(c.slots):
        want, hist = after[x][accepted[x] - 1]
        close(state[first + slot].cpu().numpy(), want, f"state of sequence {x}")
        assert np.array_equal(conv[first + slot].cpu().numpy(), hist.astype(np.float32))


@pytest.mark.parametrize("dtype,d,n_nodes,group", [("bfloat16", 128, 20, 4), ("float16", 64, 64, 3), ("float32", 64, 9, 3),
                                                   ("float32", 128, 9, 3), ("bfloat16", 256, 9, 4)])
@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_scales_that_are_not_positive(cuda_lib, dtype, d, n_nodes, group, scale):
    """The smallest score has the largest weight, or all weights are the same."""
    rng = np.random.default_rng([d, n_nodes])
    c, trees, q = case(rng, [n_nodes + 5, 400], n_nodes, 2, group, d, 16, dtype)
    call = Call(cuda_lib, c, q, trees, 2 * group)
    call.args = call.args[:-1] + (scale,)
    got = call.go().double().cpu().numpy().reshape(q.shape)
    for x, tree in enumerate(trees):
        rows = q[x * n_nodes:(x + 1) * n_nodes]
        ref = tree_cases.attention(rows, c.k[x], c.v[x], tree, scale, 0, 0)
        tol = bound(ref, rows, c.k[x], c.v[x], scale, c.dtype, weights_16bit=True)
        assert (np.abs(got[x * n_nodes:(x + 1) * n_nodes] - ref) <= tol).all()


@pytest.mark.parametrize("dtype,d,n_nodes,group", [("bfloat16", 128, 20, 4), ("float32", 64, 9, 3), ("float32", 128, 30, 1)])
def test_what_nobody_sees_may_be_anything(cuda_lib, dtype, d, n_nodes, group):
    """Infinities and NaN in cache rows in front of every window and in rows of nodes that are not there."""
    rng = np.random.default_rng(d)
    c, trees, q = case(rng, [700, 333], n_nodes, 2, group, d, 16, dtype)
    trees = [t[:n_nodes - 2] + [-2, -2] for t in trees]
    window = 50
    for x in range(2):
        for j in list(range(0, c.lens[x] - n_nodes - window + 1, 7)) + [c.lens[x] - 2, c.lens[x] - 1]:
            page = int(c.table[c.slots[x], j // 16])
            c.k_pages[page, :, j % 16] = float(rng.choice([np.inf, -np.inf, np.nan]))
            c.v_pages[page, :, j % 16] = float(rng.choice([np.inf, -np.inf, np.nan]))
    check(c, Call(cuda_lib, c, q, trees, 2 * group, window).go(), q, trees, window, 0)


def test_graphs_that_share_a_workspace(cuda_lib):
    """Two captured steps of attention and block on one workspace and tape, replayed in turn."""
    rng = np.random.default_rng(3)
    made = [case(rng, [200, 64 + 33], 20, 2, 4, 128, 16, "bfloat16") for _ in range(2)]
    calls = [Call(cuda_lib, c, q, trees, 8) for c, trees, q in made]
    calls[1].ws = calls[0].ws
    blocks = [Block(rng, [random_tree(rng, 12) for _ in range(2)], 2, 4, 128, 4, pool=2) for _ in range(2)]
    devs = [Device(cuda_lib, b) for b in blocks]
    devs[1].ws, devs[1].tape = devs[0].ws, devs[0].tape
    wanted = [plain(b)[0] for b in blocks]
    graphs = []
    for call, d in zip(calls, devs):
        c = d.c
        call.go()
        d.tree()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call.go()
            cuda_lib.gdn_block_tree(d.qkv, d.conv_w, d.conv_state, d.alpha, d.b, d.dt, d.a, d.z, d.norm_w, d.state,
                                    d.out, d.parents, c.n, c.t, c.hk, c.h, c.s, c.kernel, c.scale, c.eps, c.eps,
                                    d.tape, d.ws, **d.more)
        graphs.append(g)
    for turn in (0, 1, 0, 0, 1, 1, 0):
        calls[turn].out.fill_(7)
        devs[turn].out.fill_(7)
        graphs[turn].replay()
        torch.cuda.synchronize()
        c, trees, q = made[turn]
        check(c, calls[turn].out, q, trees, 0, 0)
        close(devs[turn].out.cpu().numpy(), wanted[turn], "the block")


def test_the_same_sequence_twice(cuda_lib):
    """Two trees on one slot: the block and the attention only read, so both have their answers."""
    rng = np.random.default_rng(9)
    c = Block(rng, [random_tree(rng, 10) for _ in range(2)], 2, 4, 128, 4, pool=2)
    c.slots = [1, 1]
    ref, _ = plain(c)
    close(Device(cuda_lib, c).tree(), ref, "the block")


def test_all_of_a_step_allocates_nothing(cuda_lib):
    rng = np.random.default_rng(11)
    calls = [Call(cuda_lib, *x) for x in
             [(c, q, trees, 8) for c, trees, q in
              [case(rng, [200, 40], 16, 2, 4, d, 16, t) for t, d in (("bfloat16", 128), ("float16", 256), ("float32", 64))]]]
    d = [Device(cuda_lib, Block(rng, [random_tree(rng, 12) for _ in range(2)], 2, 4, s, 4, pool=2)) for s in (64, 128)]
    model = Model(cuda_lib, rng, [random_tree(rng, 9) for _ in range(2)], [40, 20])
    logits = torch.randn(4, 5000, device="cuda")
    u = np.full(4, 0.5, np.float32)

    def everything():
        for call in calls:
            call.go()
        for x in d:
            x.tree()
            x.commit([1, 2])
        model.go()
        sample(cuda_lib, logits, u, temperature=[1] * 4, top_p=[0.9] * 4)
        torch.cuda.synchronize()

    everything()
    everything()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        everything()
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("spread,temperature", [(0.01, 1.0), (1.0, 4.0), (2.5, 1.3), (0.0, 1.0)])
@pytest.mark.parametrize("top_p", [0.5, 0.98, 0.9999])
def test_flat_rows(cuda_lib, dtype, spread, temperature, top_p):
    """Rows without a likely token: thousands share what is kept, and the border lies deep among them."""
    rng = np.random.default_rng([int(100 * spread), int(1e4 * top_p)])
    rows, vocab = 6, 30011
    x = torch.from_numpy((spread * rng.standard_normal((rows, vocab))).astype(np.float32)).to(getattr(torch, dtype))
    x[:, ::7] = -float("inf")
    u = rng.random(rows).astype(np.float32)
    for top_k in (0, 3000):
        more = {"top_k": [top_k] * rows} if top_k else {}
        got = sample(cuda_lib, x.cuda(), u, temperature=[temperature] * rows, top_p=[top_p] * rows, **more)
        exact = x.double().numpy()
        for r in range(rows):
            want = define(exact[r], u[r], temperature=float(np.float32(temperature)), top_p=float(np.float32(top_p)), top_k=top_k)
            assert got[r] == want, f"row {r}: token {got[r]}, not {want}"
