"""Sampling against the definition in 64 bits on the host: the tokens are equal.

The kernel's weights are good to 2^-43 of their sum and a 64-bit form's to some 2^-50, so a row
whose uniform number, or top-p border, falls within about 10^-11 of an edge could come out otherwise;
of the some 10^5 rows here that is less than one in 10^4 runs, and the seeds are fixed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = np.inf


def define(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row of logits x (64-bit)."""
    x = np.where(np.isnan(x), -INF, x)
    top = x.max()
    if top == -INF or not 0 <= temperature < INF or np.isnan(top_p) or np.isnan(min_p):
        return -1
    order = np.argsort(-x, kind="stable")
    s = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(s == top, 1.0, np.exp((s - top) / (temperature if temperature > 0 else 1.0)))
    keep = s > -INF
    if 0 < top_k < len(x):
        keep &= np.arange(len(x)) < top_k
    w = np.where(keep, w, 0.0)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep &= before < top_p * w.sum()
    if min_p > 0:
        keep &= w >= min_p
    keep[0] = True
    if temperature == 0:
        keep[1:] = False
    by_index = np.zeros(len(x))
    by_index[order] = np.where(keep, w, 0.0)
    cdf = np.cumsum(by_index)
    u = np.float32(0 if np.isnan(u) else min(max(u, 0.0), np.float32(1 - 2.0 ** -24)))
    return int(np.searchsorted(cdf, np.float64(u) * cdf[-1], side="right"))


def typed(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(getattr(torch, dtype))


def f32(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def sample(gdn, logits, u, per_set=1, err=None, **settings):
    """logits: a CUDA tensor [rows][vocab]."""
    rows, vocab = logits.shape
    tokens = torch.full((rows + 1,), 77, dtype=torch.int32, device="cuda")
    args = {k: torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda() if k == "top_k" else f32(v)
            for k, v in settings.items()}
    gdn.gdn_sample(logits, f32(u), tokens, rows, vocab, rows_per_set=per_set, err_count=err, **args)
    got = tokens.tolist()
    assert got[-1] == 77
    return got[:-1]


def check(gdn, x, u, dtype="float32", per_set=1, logits=None, **settings):
    t = typed(x, dtype)
    got = sample(gdn, t.cuda() if logits is None else logits, u, per_set, **settings)
    exact = t.double().numpy()
    for r in range(len(exact)):
        # 32-bit settings, as the call takes them
        mine = {k: float(np.float32(v[r // per_set])) if k != "top_k" else int(v[r // per_set]) for k, v in settings.items()}
        want = define(exact[r], u[r], **mine)
        assert got[r] == want, f"row {r}: token {got[r]}, not {want} ({mine}, u {u[r]})"
    return got


def settings_of(rng, kind, n):
    out = {"temperature": rng.choice([0.3, 0.7, 1.0, 1.5, 4.0], n)}
    if kind == "greedy":
        out["temperature"] = np.zeros(n)
    if kind in ("top_k", "all"):
        out["top_k"] = np.exp(rng.uniform(0, np.log(3000), n)).astype(int)
    if kind in ("top_p", "all"):
        out["top_p"] = rng.choice([0.0, 1e-6, 0.1, 0.5, 0.9, 0.95, 0.999, 1.0], n)
    if kind in ("min_p", "all"):
        out["min_p"] = rng.choice([0.0, 1e-5, 0.02, 0.1, 0.7, 1.0, 1.5], n)
    return out


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 31, 33, 257, 1000, 4099, 32768, 50257, 131072])
@pytest.mark.parametrize("kind", ["greedy", "free", "top_k", "top_p", "min_p", "all"])
def test_tokens(cuda_lib, dtype, vocab, kind):
    rng = np.random.default_rng([vocab, len(kind)])
    rows = 24 if vocab < 5000 else 8
    x = rng.standard_normal((rows, vocab)) * rng.choice([0.1, 1, 3, 10], (rows, 1))
    check(cuda_lib, x, rng.random(rows).astype(np.float32), dtype, **settings_of(rng, kind, rows))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("kind", ["greedy", "free", "top_k", "top_p", "min_p", "all"])
@pytest.mark.parametrize("levels", [1, 2, 5])
def test_ties(cuda_lib, dtype, kind, levels):
    """Few different logits: what is kept ends among equals, which go by their index; sums are whole
    numbers where there is one level, and uniform numbers fall on the borders themselves."""
    rng = np.random.default_rng([levels, len(kind)])
    rows, vocab = 40, 6000
    x = rng.choice(np.linspace(-3, 2, levels), (rows, vocab))
    u = rng.integers(0, vocab, rows) / vocab if levels == 1 else rng.random(rows)
    settings = settings_of(rng, kind, rows)
    if levels == 1 and kind == "top_p":
        settings["top_p"] = rng.choice([0.25, 0.5, 0.125, 0.75], rows)
    check(cuda_lib, x, u.astype(np.float32), dtype, **settings)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kind", ["greedy", "free", "top_k", "top_p", "min_p", "all"])
def test_masked_and_odd_logits(cuda_lib, dtype, kind):
    """Banned tokens, rows with one token left, with none, with infinities, NaN, both zeros."""
    rng = np.random.default_rng(len(kind))
    vocab = 3001
    x = rng.standard_normal((16, vocab))
    x[0, rng.random(vocab) < 0.9] = -INF
    x[1] = -INF
    x[1, 1234] = -5.0
    x[2] = -INF
    x[3] = np.nan
    x[4, ::2] = np.nan
    x[5, 100] = INF
    x[6, [7, 70, 700]] = INF
    x[7] = INF
    x[8] = np.where(rng.random(vocab) < 0.5, 0.0, -0.0)
    x[9] = -30000.0
    x[9, 5] = 30000.0
    x[10, :-1] = -INF
    x[11, 1:] = -INF
    x[12] = 1e-30 * x[12]
    x[13] = 60000.0
    u = rng.random(16)
    u[14], u[15] = 0.0, 1 - 2.0 ** -24
    got = check(cuda_lib, x, u.astype(np.float32), dtype, **settings_of(rng, kind, 16))
    assert got[2] == got[3] == -1 and got[1] == 1234 and got[5] == 100 and got[10] == vocab - 1


@pytest.mark.parametrize("temperature", [1e-30, 1e-6, 100.0, 1e20])
def test_temperatures(cuda_lib, temperature):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 9000))
    check(cuda_lib, x, rng.random(6).astype(np.float32), temperature=[temperature] * 6, top_p=[0.9] * 6)


def test_uniform_numbers_out_of_range(cuda_lib):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 500))
    check(cuda_lib, x, np.array([-1, 1.0, 2.0, np.nan, INF, -INF], np.float32))


def test_settings_that_are_not_valid(cuda_lib):
    rng = np.random.default_rng(3)
    x = typed(rng.standard_normal((6, 500)), "float32").cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nan = np.nan
    got = sample(cuda_lib, x, np.full(6, 0.5), err=err, temperature=[-1, INF, nan, 1, 1, 1],
                 top_p=[1, 1, 1, nan, 1, 1], min_p=[0, 0, 0, 0, nan, 0])
    assert got[:5] == [-1] * 5 and got[5] >= 0 and err.item() == 5


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("vocab,stride,offset", [(1001, 1003, 0), (1001, 1001, 1), (4096, 4103, 3), (50001, 50007, 5), (5, 9, 2)])
def test_slices_and_alignments(cuda_lib, dtype, vocab, stride, offset):
    """Rows that are slices of wider ones, beginning anywhere; what lies beside them is larger."""
    rng = np.random.default_rng([vocab, offset])
    rows = 9
    x = 2 * rng.standard_normal((rows, vocab))
    wide = torch.full((rows * stride + offset,), 50.0, dtype=getattr(torch, dtype), device="cuda")
    view = wide[offset:].view(rows, stride)[:, :vocab]
    view.copy_(typed(x, dtype))
    u = rng.random(rows).astype(np.float32)
    check(cuda_lib, x, u, dtype, logits=view, top_p=[0.95] * rows)
    check(cuda_lib, x, u, dtype, logits=view)


def test_settings_of_sets_of_rows(cuda_lib):
    rng = np.random.default_rng(5)
    rows, per_set = 23, 5
    x = 3 * rng.standard_normal((rows, 2000))
    check(cuda_lib, x, rng.random(rows).astype(np.float32), per_set=per_set, **settings_of(rng, "all", 5))


def test_many_rows(cuda_lib):
    """More rows than clusters fit at once, by every number of CTAs a row."""
    rng = np.random.default_rng(6)
    for rows, vocab in ((700, 1500), (300, 9001), (70, 40000)):
        x = 2 * rng.standard_normal((rows, vocab))
        check(cuda_lib, x, rng.random(rows).astype(np.float32), "bfloat16", **settings_of(rng, "all", rows))


@pytest.mark.parametrize("dtype,vocab", [("float32", 390000), ("bfloat16", 500001)])
def test_largest_vocabularies(cuda_lib, dtype, vocab):
    rng = np.random.default_rng(7)
    x = 2 * rng.standard_normal((3, vocab))
    check(cuda_lib, x, rng.random(3).astype(np.float32), dtype, temperature=[1, 0.8, 1.2], top_p=[1, 0.9, 0.5])


def test_shares_are_the_weights(cuda_lib):
    """Uniform numbers spread evenly: a token comes out as often as its weight says, but for one."""
    rng = np.random.default_rng(8)
    n, vocab = 4000, 37
    x = rng.standard_normal(vocab).astype(np.float32)
    logits = torch.from_numpy(np.tile(x, (n, 1))).cuda()
    got = np.bincount(sample(cuda_lib, logits, (np.arange(n) + 0.5) / n), minlength=vocab)
    w = np.exp(x.astype(np.float64) - x.max())
    assert np.abs(got - n * w / w.sum()).max() <= 1.0


@pytest.mark.parametrize("dtype,temperature,top_p", [("float32", 1.3, 1.0), ("float32", 0.7, 0.97), ("bfloat16", 1.0, 1.0)])
def test_many_numbers_over_a_flat_row(cuda_lib, dtype, temperature, top_p):
    """Thousands of uniform numbers over one row whose tokens are all unlikely, so that errors of some
    10^-7 in the weights or their sum would show."""
    rng = np.random.default_rng(10)
    n, vocab = 4000, 50021
    t = typed(1.5 * rng.standard_normal(vocab), dtype)
    u = rng.random(n).astype(np.float32)
    got = sample(cuda_lib, t.cuda().repeat(n, 1), u, temperature=[temperature] * n, top_p=[top_p] * n)
    x = t.double().numpy()
    w = np.exp((x - x.max()) / np.float64(np.float32(temperature)))
    order = np.argsort(-x, kind="stable")
    before = np.cumsum(w[order]) - w[order]
    kept = np.zeros(vocab, bool)
    kept[order] = before < np.float64(np.float32(top_p)) * w.sum() if top_p < 1 else True
    cdf = np.cumsum(np.where(kept, w, 0.0))
    assert got == np.searchsorted(cdf, u.astype(np.float64) * cdf[-1], side="right").tolist()


def test_captured_and_replayed_and_on_two_streams(cuda_lib):
    rng = np.random.default_rng(9)
    rows, vocab = 20, 20011
    logits = torch.zeros(rows, vocab, device="cuda", dtype=torch.bfloat16)
    u, tokens = torch.zeros(rows, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    p = torch.full((rows,), 0.9, device="cuda")
    call = lambda **more: cuda_lib.gdn_sample(logits, u, tokens, rows, vocab, top_p=p, **more)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for replay in (graph.replay, lambda: call(stream=side.cuda_stream)):
        side = torch.cuda.Stream()
        x = typed(2 * rng.standard_normal((rows, vocab)), "bfloat16")
        numbers = rng.random(rows).astype(np.float32)
        logits.copy_(x)
        u.copy_(f32(numbers))
        torch.cuda.synchronize()
        replay()
        torch.cuda.synchronize()
        exact = x.double().numpy()
        assert tokens.tolist() == [define(exact[r], numbers[r], top_p=float(np.float32(0.9))) for r in range(rows)]
