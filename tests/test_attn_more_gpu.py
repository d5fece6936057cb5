"""Shapes of the attention calls that the other files leave out (fp32 units of 8 and 16 rows with
heads of 256, drafts of several tokens in 16-bit types with narrow and wide heads), against the
plain form in 64 bits; and that no call allocates device memory."""
import numpy as np
import pytest

from tests.attn_cases import Cache
from tests.test_attn_decode_gpu import run as decode
from tests.test_attn_prefill_gpu import run as prefill
from tests.test_pages_gpu import Device, Model

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_tokens,group", [(1, 7), (1, 16), (2, 6), (3, 5), (1, 40)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (75, 3)])
def test_fp32_units_of_many_rows(cuda_lib, d, n_tokens, group, window, sinks):
    rng = np.random.default_rng([d, n_tokens, group])
    lens = [n_tokens, 31, 32, 33, 500, 0, 4000]
    c = Cache(torch, rng, lens, 2, d, 16, "float32")
    counts = [n_tokens] * len(lens)
    q = c.queries(rng, counts, 2 * group)
    c.check(decode(cuda_lib, c, q, n_tokens, 2 * group, window, sinks), q, counts, d ** -0.5, window, sinks)
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("dtype,d", [("bfloat16", 64), ("float16", 64), ("bfloat16", 256), ("float16", 256)])
@pytest.mark.parametrize("n_tokens,group", [(3, 1), (4, 4), (5, 3), (17, 2), (64, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
def test_drafts_of_16_bit_types(cuda_lib, dtype, d, n_tokens, group, window, sinks):
    rng = np.random.default_rng([d, n_tokens, group])
    lens = [n_tokens, 1, 64, 64 + n_tokens - 1, 700, 0, 129]
    c = Cache(torch, rng, lens, 2, d, 32, dtype)
    counts = [n_tokens] * len(lens)
    q = c.queries(rng, counts, 2 * group)
    c.check(decode(cuda_lib, c, q, n_tokens, 2 * group, window, sinks), q, counts, d ** -0.5, window, sinks)
    cuda_lib.gdn_device_error()


def test_no_call_allocates(cuda_lib):
    """The device's free memory is the same after calls whose kernels have run before. (torch holds
    what the tests' own tensors need from the first round on.)"""
    rng = np.random.default_rng(1)
    lens, counts = [400, 33], [40, 33]
    caches = [Cache(torch, rng, lens, 2, d, 16, t) for t, d in
              (("float32", 64), ("bfloat16", 128), ("float16", 256))]
    asked = [(c, c.queries(rng, [1, 1], 4), c.queries(rng, counts, 4)) for c in caches]

    def everything():
        for c, q, prompt in asked:
            decode(cuda_lib, c, q, 1, 4)
            prefill(cuda_lib, c, prompt, counts, 4)
            k = torch.zeros(2, 2, c.d, dtype=c.k_pages.dtype, device="cuda")
            cuda_lib.gdn_kv_append(k, k, c.k_pages.clone(), c.v_pages.clone(), c.d_table, c.d_lens,
                                   None, 2, 2, 2, c.d, 16, c.n_pages, c.max_pages, slots=c.d_slots,
                                   pool=c.pool)
        d = Device(cuda_lib, Model(np.random.default_rng(2), 6, 20, 8, 4))
        d.reserve([0, 1], [13, 16])
        d.fork([0, 1], [2, 3])
        d.truncate([0, 2], [3, 0])
        d.compact()
        cuda_lib.gdn_pages_copy(d.pages, d.ints([0]), d.ints([9]), 1, 3, 20, 48)
        torch.cuda.synchronize()

    everything()
    everything()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        everything()
    assert torch.cuda.mem_get_info()[0] == free
