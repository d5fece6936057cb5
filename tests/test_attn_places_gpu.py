"""Where a call's data lies and runs: pages past 2^32 bytes of their plane, streams other than
the current one, replays of a captured call."""
import numpy as np
import pytest

from tests.attn_cases import Cache
from tests.test_attn_decode_gpu import run as decode
from tests.test_attn_prefill_gpu import run as prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def move_up(c, past_bytes):
    """The cache's pages at the end of planes of more than past_bytes bytes."""
    first = past_bytes // (c.k_pages[0].numel() * c.k_pages.element_size()) + 1
    for name in ("k_pages", "v_pages"):
        small = getattr(c, name)
        big = torch.empty((first + c.n_pages, *small.shape[1:]), dtype=small.dtype, device="cuda")
        big[first:] = small
        setattr(c, name, big)
    c.n_pages += first
    c.table = np.where(c.table >= 0, c.table + first, c.table).astype(np.int32)
    c.d_table = torch.from_numpy(c.table).cuda()


@pytest.mark.parametrize("dtype,d,ps", [("bfloat16", 128, 256), ("float16", 64, 16), ("float32", 128, 64)])
def test_pages_past_32_bits(cuda_lib, dtype, d, ps):
    rng = np.random.default_rng([d, ps])
    lens, scale = [300, 77], 1.0 / np.sqrt(d)
    c = Cache(torch, rng, lens, 2, d, ps, dtype)
    move_up(c, 1 << 32)
    q = c.queries(rng, [1, 1], 6)
    c.check(decode(cuda_lib, c, q, 1, 6), q, [1, 1], scale, 0, 0)
    counts = [40, 77]
    q = c.queries(rng, counts, 6)
    c.check(prefill(cuda_lib, c, q, counts, 6), q, counts, scale, 0, 0, weights_16bit=True)
    # the last rows written once more, from elsewhere
    k = torch.randn(2, 2, d, device="cuda").to(c.k_pages.dtype)
    v = torch.randn(2, 2, d, device="cuda").to(c.k_pages.dtype)
    cuda_lib.gdn_kv_append(k, v, c.k_pages, c.v_pages, c.d_table, c.d_lens, None, 2, 2, 2, d, ps,
                           c.n_pages, c.max_pages, slots=c.d_slots, pool=c.pool)
    for i, n in enumerate(lens):
        page, row = int(c.table[c.slots[i], (n - 1) // ps]), (n - 1) % ps
        assert torch.equal(c.k_pages[page, :, row], k[i]) and torch.equal(c.v_pages[page, :, row], v[i])


def test_copy_past_32_bits(cuda_lib):
    page_bytes, n_pages = 1 << 16, (1 << 16) + 9
    pages = torch.zeros(2, n_pages, page_bytes, dtype=torch.uint8, device="cuda")
    pages[:, :4] = torch.randint(1, 256, (2, 4, page_bytes), device="cuda", dtype=torch.int32).to(torch.uint8)
    ints = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    cuda_lib.gdn_pages_copy(pages, ints(0, 1, 2, 3), ints(n_pages - 1, n_pages - 3, 5, 1 << 16), 4, 2,
                            n_pages, page_bytes)
    for s, t in ((0, n_pages - 1), (1, n_pages - 3), (2, 5), (3, 1 << 16)):
        assert torch.equal(pages[:, s], pages[:, t])
    assert pages.any(-1).sum().item() == 16


@pytest.mark.parametrize("dtype,d", [("bfloat16", 64), ("float16", 256), ("float32", 128)])
def test_prompt_on_a_side_stream_and_replayed(cuda_lib, dtype, d):
    """Append and prompt attention behind one another on a stream of their own, from slices of a
    wider row, and captured: replays see other rows in the same places."""
    rng = np.random.default_rng(d)
    counts, hq = [70, 1, 33], 4
    c = Cache(torch, rng, counts, 2, d, 16, dtype)
    total, n = sum(counts), len(counts)
    rows = torch.zeros(total, hq + 4, d, dtype=c.k_pages.dtype, device="cuda")
    out = torch.zeros(total, hq, d, dtype=c.k_pages.dtype, device="cuda")
    cu = torch.tensor([0, 70, 71, 104], dtype=torch.int32, device="cuda")
    books = (c.k_pages, c.v_pages, c.d_table, c.d_lens)
    pages = dict(slots=c.d_slots, pool=c.pool)

    def call():
        cuda_lib.gdn_kv_append(rows[:, hq:hq + 2], rows[:, hq + 2:], *books, cu, n, total, 2, d, 16,
                               c.n_pages, c.max_pages, **pages)
        cuda_lib.gdn_attn_prefill(rows[:, :hq], *books, out, cu, n, total, 70, hq, 2, d, 16, c.n_pages,
                                  c.max_pages, 0, 0, 1.0 / np.sqrt(d), **pages)

    def fill():
        q = c.queries(rng, counts, hq)
        k, v = c.typed(rng.standard_normal((total, 2, d))), c.typed(rng.standard_normal((total, 2, d)))
        rows.copy_(c.dev(np.concatenate([q, k, v], 1)))
        c.k, c.v = np.split(k, [70, 71]), np.split(v, [70, 71])
        return q

    q = fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    c.check(out, q, counts, 1.0 / np.sqrt(d), 0, 0, weights_16bit=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        q = fill()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, q, counts, 1.0 / np.sqrt(d), 0, 0, weights_16bit=True)
