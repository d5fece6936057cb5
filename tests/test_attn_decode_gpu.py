"""Attention of new tokens over the paged cache, against the plain form in 64 bits."""
import numpy as np
import pytest

from tests.attn_cases import Cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def run(gdn, cache, q, n_tokens, hq, window=0, sinks=0, scale=None, ws_fill=0xFF, slots=True,
        err=None, wide=False, out_fill=float("nan")):
    """One call; q packed [n * n_tokens][hq][d] (64-bit numpy). Returns out (device)."""
    d, n = cache.d, len(cache.lens)
    qd = cache.dev(q)
    if wide:  # q as a slice of a wider row
        row = torch.zeros(n * n_tokens, hq + 2 * cache.hkv, d, dtype=qd.dtype, device="cuda")
        row[:, :hq] = qd
        qd = row[:, :hq]
    out = torch.full((n * n_tokens, hq, d), out_fill, dtype=qd.dtype, device="cuda")
    size = gdn.gdn_attn_decode_workspace_size(n, n_tokens, hq, cache.hkv, d)
    ws = torch.full((size,), ws_fill, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_decode(qd, cache.k_pages, cache.v_pages, cache.d_table, cache.d_lens, out, n,
                        n_tokens, hq, cache.hkv, d, cache.ps, cache.n_pages, cache.max_pages,
                        window, sinks, cache_scale(cache) if scale is None else scale, ws,
                        slots=cache.d_slots if slots else None, pool=cache.pool, err_count=err)
    return out


def cache_scale(cache):
    return 1.0 / np.sqrt(cache.d)


LENS = [1, 0, 2, 7, 63, 64, 65, 200, 1000]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,group", [(1, 1), (2, 3), (1, 8), (5, 4)])
def test_types_and_heads(cuda_lib, dtype, d, hkv, group):
    rng = np.random.default_rng([d, hkv, group, len(dtype)])
    c = Cache(torch, rng, LENS, hkv, d, 16, dtype, pool=12)
    q = c.queries(rng, [1] * len(LENS), hkv * group)
    out = run(cuda_lib, c, q, 1, hkv * group)
    c.check(out, q, [1] * len(LENS), cache_scale(c), 0, 0)
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_page_sizes(cuda_lib, ps, dtype):
    rng = np.random.default_rng(ps)
    lens = [ps - 1, ps, ps + 1, 3 * ps, 5, 777]
    c = Cache(torch, rng, lens, 2, 128, ps, dtype)
    q = c.queries(rng, [1] * len(lens), 4)
    c.check(run(cuda_lib, c, q, 1, 4, wide=True), q, [1] * len(lens), cache_scale(c), 0, 0)


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 64), (100, 3), (5000, 2),
                                          (33, 700), (0, 9)])
def test_windows_and_sinks(cuda_lib, dtype, window, sinks):
    """Pages wholly between the sinks and the window are gone: their ids point nowhere."""
    rng = np.random.default_rng([window, sinks])
    lens = [1, 16, 17, 90, 640, 1001]
    gone = [(sinks, max(sinks, n - window)) if window else (0, 0) for n in lens]
    c = Cache(torch, rng, lens, 2, 64, 16, dtype, evicted=gone)
    q = c.queries(rng, [1] * len(lens), 6)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(cuda_lib, c, q, 1, 6, window, sinks, err=err)
    c.check(out, q, [1] * len(lens), cache_scale(c), window, sinks)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n_tokens,group", [(2, 1), (4, 4), (5, 3), (4, 8), (17, 2), (3, 16), (2, 20)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_draft_tokens(cuda_lib, dtype, n_tokens, group, window, sinks):
    """Several new tokens, each seeing one key more; a sequence shorter than the draft has
    rows before position 0, which see nothing."""
    rng = np.random.default_rng([n_tokens, group, window])
    lens = [n_tokens, 1, 64, 64 + n_tokens - 1, 300, 0]
    c = Cache(torch, rng, lens, 2, 128, 16, dtype)
    counts = [n_tokens] * len(lens)
    q = c.queries(rng, counts, 2 * group)
    out = run(cuda_lib, c, q, n_tokens, 2 * group, window, sinks)
    c.check(out, q, counts, cache_scale(c), window, sinks)


@pytest.mark.parametrize("dtype,d,group", [("bfloat16", 128, 4), ("float32", 64, 2),
                                           ("float16", 256, 8)])
@pytest.mark.parametrize("lens", [[20000], [1] * 700, [9000, 1, 1, 5000, 30]])
def test_split_and_joined(cuda_lib, dtype, d, group, lens):
    """One long sequence over all CTAs, many short ones, and a mix; twice for the same bits, on
    a workspace full of ones and one full of zeros."""
    rng = np.random.default_rng(len(lens))
    c = Cache(torch, rng, lens, 1, d, 64, dtype)
    q = c.queries(rng, [1] * len(lens), group)
    a = run(cuda_lib, c, q, 1, group, ws_fill=0xFF)
    b = run(cuda_lib, c, q, 1, group, ws_fill=0)
    c.check(a, q, [1] * len(lens), cache_scale(c), 0, 0)
    assert torch.equal(a, b)
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_large_scores(cuda_lib, dtype):
    """Scores of both signs in the hundreds: one key takes nearly all the weight."""
    rng = np.random.default_rng(5)
    lens = [300, 40]
    c = Cache(torch, rng, lens, 1, 64, 16, dtype)
    q = c.queries(rng, [1, 1], 2)
    for scale in (4.0, -4.0, 0.0):
        c.check(run(cuda_lib, c, q, 1, 2, scale=scale), q, [1, 1], scale, 0, 0)


def test_skipped_sequences_and_bad_pages(cuda_lib):
    """A slot or length out of range leaves the sequence's rows alone and counts it; a visible
    page id out of range hides its keys."""
    rng = np.random.default_rng(6)
    lens = [70, 80, 90, 100]
    c = Cache(torch, rng, lens, 2, 64, 16, "bfloat16", pool=6)
    q = c.queries(rng, [1] * 4, 4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = c.slots.copy()
    c.d_slots[0] = 6
    c.d_lens[int(slots[1])] = 16 * c.max_pages + 1
    c.d_table[int(slots[2]), 2] = c.n_pages  # keys 32 .. 47 of sequence 2
    out = run(cuda_lib, c, q, 1, 4, err=err, out_fill=7.0)
    assert (out[0] == 7).all() and (out[1] == 7).all()
    assert err.item() >= 3
    keep = np.r_[0:32, 48:90]
    c.k[2], c.v[2], c.lens[2] = c.k[2][keep], c.v[2][keep], len(keep)
    c.k[:2], c.v[:2], c.lens[:2] = [], [], []
    c.check(out[2:], q[2:], [1, 1], cache_scale(c), 0, 0)


def test_other_stream_and_graph(cuda_lib):
    """On a stream of its own, and captured: replays see the cache grow."""
    rng = np.random.default_rng(7)
    lens = [500, 33, 260]
    c = Cache(torch, rng, lens, 2, 128, 32, "bfloat16")
    q = c.queries(rng, [1] * 3, 8)
    want = run(cuda_lib, c, q, 1, 8)
    qd = c.dev(q)
    out = torch.zeros_like(want)
    ws = torch.empty(cuda_lib.gdn_attn_decode_workspace_size(3, 1, 8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    call = lambda: cuda_lib.gdn_attn_decode(  # noqa: E731
        qd, c.k_pages, c.v_pages, c.d_table, c.d_lens, out, 3, 1, 8, 2, 128, c.ps, c.n_pages,
        c.max_pages, 0, 0, cache_scale(c), ws, slots=c.d_slots, pool=c.pool)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for shorter in (0, 1, 17):
        c.d_lens.copy_(torch.from_numpy(c.kv_lens) - shorter)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        cut = Cache.__new__(Cache)
        cut.__dict__.update(c.__dict__)
        cut.lens = [n - shorter for n in lens]
        cut.k = [x[:n] for x, n in zip(c.k, cut.lens)]
        cut.v = [x[:n] for x, n in zip(c.v, cut.lens)]
        cut.check(out, q, [1] * 3, cache_scale(c), 0, 0)
