"""Attention of ragged prompts over the paged cache, against the plain form in 64 bits."""
import numpy as np
import pytest

from tests.attn_cases import Cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def run(gdn, cache, q, counts, hq, window=0, sinks=0, scale=None, cu=None, err=None, wide=False,
        out_fill=float("nan"), max_tokens=None):
    d, n, total = cache.d, len(counts), sum(counts)
    qd = cache.dev(q)
    if wide:
        row = torch.zeros(total, hq + 2 * cache.hkv, d, dtype=qd.dtype, device="cuda")
        row[:, :hq] = qd
        qd = row[:, :hq]
    out = torch.full((total, hq, d), out_fill, dtype=qd.dtype, device="cuda")
    if cu is None:
        cu = np.concatenate([[0], np.cumsum(counts)])
    d_cu = torch.from_numpy(np.asarray(cu, np.int32)).cuda()
    size = gdn.gdn_attn_prefill_workspace_size(n, total, hq, cache.hkv, d)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_prefill(qd, cache.k_pages, cache.v_pages, cache.d_table, cache.d_lens, out, d_cu,
                         n, total, max(counts) if max_tokens is None else max_tokens, hq,
                         cache.hkv, d, cache.ps, cache.n_pages, cache.max_pages, window, sinks,
                         1.0 / np.sqrt(d) if scale is None else scale, ws, slots=cache.d_slots,
                         pool=cache.pool, err_count=err)
    return out


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,group", [(2, 1), (1, 3), (1, 8), (2, 5), (1, 20)])
def test_types_and_heads(cuda_lib, dtype, d, hkv, group):
    """Fresh prompts and chunks that follow a history, from one token on."""
    rng = np.random.default_rng([d, hkv, group])
    counts = [1, 40, 3, 130, 0, 17]
    lens = [1, 40, 70, 200, 9, 300]
    c = Cache(torch, rng, lens, hkv, d, 16, dtype, pool=8)
    q = c.queries(rng, counts, hkv * group)
    out = run(cuda_lib, c, q, counts, hkv * group, wide=True)
    c.check(out, q, counts, 1.0 / np.sqrt(d), 0, 0, weights_16bit=True)
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_page_sizes(cuda_lib, ps, dtype):
    rng = np.random.default_rng(ps)
    counts, lens = [33, 64, 5, 150], [33, 64 + ps, 300, 150]
    c = Cache(torch, rng, lens, 2, 128, ps, dtype)
    q = c.queries(rng, counts, 4)
    c.check(run(cuda_lib, c, q, counts, 4), q, counts, 128 ** -0.5, 0, 0, weights_16bit=True)


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 64), (100, 3), (5000, 2),
                                          (33, 400), (0, 9), (300, 0)])
def test_windows_and_sinks(cuda_lib, dtype, window, sinks):
    """Pages that no new position sees are gone: their ids point nowhere."""
    rng = np.random.default_rng([window, sinks])
    counts, lens = [200, 30, 1, 64], [200, 700, 513, 64]
    gone = [(sinks, max(sinks, n - m - window + 1)) if window else (0, 0)
            for m, n in zip(counts, lens)]
    c = Cache(torch, rng, lens, 1, 64, 16, dtype, evicted=gone)
    q = c.queries(rng, counts, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(cuda_lib, c, q, counts, 2, window, sinks, err=err)
    c.check(out, q, counts, 0.125, window, sinks, weights_16bit=True)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_long_prompt(cuda_lib, dtype):
    rng = np.random.default_rng(11)
    counts, lens = [90, 300], [2500, 1111]
    c = Cache(torch, rng, lens, 1, 128, 64, dtype)
    q = c.queries(rng, counts, 4)
    a = run(cuda_lib, c, q, counts, 4)
    c.check(a, q, counts, 128 ** -0.5, 0, 0, weights_16bit=True)
    assert torch.equal(a, run(cuda_lib, c, q, counts, 4))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_large_scores(cuda_lib, dtype):
    rng = np.random.default_rng(5)
    c = Cache(torch, rng, [300, 40], 1, 64, 16, dtype)
    q = c.queries(rng, [150, 40], 2)
    for scale in (4.0, -4.0, 0.0):
        c.check(run(cuda_lib, c, q, [150, 40], 2, scale=scale), q, [150, 40], scale, 0, 0,
                weights_16bit=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_more_new_tokens_than_positions(cuda_lib, dtype):
    """Rows before position 0 see nothing: zeros."""
    rng = np.random.default_rng(8)
    c = Cache(torch, rng, [3, 0], 1, 64, 16, dtype)
    q = c.queries(rng, [7, 2], 2)
    c.check(run(cuda_lib, c, q, [7, 2], 2), q, [7, 2], 0.125, 0, 0, weights_16bit=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_skipped_sequences_and_bad_pages(cuda_lib, dtype):
    rng = np.random.default_rng(6)
    counts, lens = [70, 80, 20, 100], [70, 80, 90, 100]
    c = Cache(torch, rng, lens, 2, 64, 16, dtype, pool=6)
    q = c.queries(rng, counts, 4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = c.slots.copy()
    c.d_slots[0] = -1
    c.d_lens[int(slots[1])] = -5
    c.d_table[int(slots[2]), 2] = -1  # keys 32 .. 47 of sequence 2
    out = run(cuda_lib, c, q, counts, 4, err=err, out_fill=7.0)
    assert (out[:150] == 7).all()
    assert err.item() >= 3
    keep = np.r_[0:32, 48:90]
    c.k[2], c.v[2], c.lens[2] = c.k[2][keep], c.v[2][keep], len(keep)
    c.k[:2], c.v[:2], c.lens[:2] = [], [], []
    c.check(out[150:], q[150:], counts[2:], 0.125, 0, 0, weights_16bit=True)


def test_invalid_ranges_are_skipped(cuda_lib):
    rng = np.random.default_rng(9)
    counts, lens = [20, 30, 10], [20, 30, 10]
    c = Cache(torch, rng, lens, 1, 64, 16, "bfloat16")
    q = c.queries(rng, counts, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the second sequence is longer than max_tokens
    out = run(cuda_lib, c, q, counts, 2, err=err, out_fill=7.0, max_tokens=20)
    assert err.item() == 1 and (out[20:50] == 7).all()
    got = torch.cat([out[:20], out[50:]])
    del c.k[1], c.v[1], c.lens[1]
    c.check(got, np.concatenate([q[:20], q[50:]]), [20, 10], 0.125, 0, 0, weights_16bit=True)


def test_one_token_prompts_match_decode(cuda_lib):
    """A prompt chunk of one token is the decode call's question."""
    from tests.test_attn_decode_gpu import run as decode
    rng = np.random.default_rng(10)
    lens = [400, 7, 64]
    c = Cache(torch, rng, lens, 2, 128, 16, "float16")
    q = c.queries(rng, [1] * 3, 8)
    c.check(run(cuda_lib, c, q, [1] * 3, 8), q, [1] * 3, 128 ** -0.5, 0, 0, weights_16bit=True)
    c.check(decode(cuda_lib, c, q, 1, 8), q, [1] * 3, 128 ** -0.5, 0, 0)


@pytest.mark.parametrize("dtype,d", [("float16", 64), ("bfloat16", 128), ("float16", 256),
                                     ("float32", 64)])
@pytest.mark.parametrize("n_seqs", [37, 300])
def test_many_sequences(cuda_lib, dtype, d, n_seqs):
    """Ragged batches below and above the size that is put in order of length, lengths on both
    sides of the tiles' edges, sequences without new tokens among them; the same bits twice."""
    rng = np.random.default_rng([n_seqs, d])
    counts = [int(x) for x in rng.choice([0, 1, 2, 31, 32, 33, 64, 65, 127, 128, 129], n_seqs)]
    lens = [m + int(rng.choice([0, 0, 1, 100, 128, 300])) for m in counts]
    c = Cache(torch, rng, lens, 1, d, 32, dtype, pool=n_seqs + 5)
    q = c.queries(rng, counts, 4)
    a = run(cuda_lib, c, q, counts, 4, 70, 3)
    c.check(a, q, counts, d ** -0.5, 70, 3, weights_16bit=True)
    assert torch.equal(a, run(cuda_lib, c, q, counts, 4, 70, 3))
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype,d,group", [("bfloat16", 64, 1), ("bfloat16", 128, 4),
                                           ("float16", 128, 128), ("float16", 256, 7)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 1), (130, 200), (256, 3)])
def test_row_tiles_at_the_edges(cuda_lib, dtype, d, group, window, sinks):
    """Row tiles whose window, sinks and diagonal fall into different key tiles, chunk by chunk."""
    rng = np.random.default_rng([d, group, window])
    counts = [260, 129, 70]
    lens = [260, 640, 400]
    c = Cache(torch, rng, lens, 1, d, 16, dtype)
    q = c.queries(rng, counts, group)
    out = run(cuda_lib, c, q, counts, group, window, sinks)
    c.check(out, q, counts, d ** -0.5, window, sinks, weights_16bit=True)
    cuda_lib.gdn_device_error()
