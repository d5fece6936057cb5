"""The attention calls' watchdog flags: a bounded wait that runs out (on an mbarrier armed for
bytes no copy brings, a millisecond here) is reported once, its guarded write does not happen,
and the calls work afterwards. Nothing faults, traps or hangs."""
import numpy as np
import pytest

from tests.attn_cases import Cache
from tests.test_attn_decode_gpu import run as decode
from tests.test_attn_prefill_gpu import run as prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GDN_OK, GDN_ERR_DEVICE = 0, 6


def status(gdn):
    return gdn.library().gdn_device_error(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("armed", [0, 1, 2, 3])
def test_a_wait_that_runs_out_is_reported(cuda_lib, armed):
    assert status(cuda_lib) == GDN_OK  # nothing pending from earlier work
    out = torch.full((3,), 5.0, device="cuda")
    cuda_lib.gdn_selftest_attn_wait(armed, 1000, out)
    assert status(cuda_lib) == (GDN_ERR_DEVICE if armed else GDN_OK)
    assert status(cuda_lib) == GDN_OK  # read and cleared
    assert out.tolist() == [5.0 if armed & 1 else 1.0, 5.0 if armed & 2 else 1.0, 5.0]


def test_the_calls_work_afterwards(cuda_lib):
    cuda_lib.gdn_selftest_attn_wait(3, 1000, torch.zeros(2, device="cuda"))
    assert status(cuda_lib) == GDN_ERR_DEVICE
    rng = np.random.default_rng(0)
    lens, counts = [300, 17], [40, 17]
    c = Cache(torch, rng, lens, 2, 64, 16, "bfloat16")
    q = c.queries(rng, [1, 1], 4)
    c.check(decode(cuda_lib, c, q, 1, 4), q, [1, 1], 0.125, 0, 0)
    q = c.queries(rng, counts, 4)
    c.check(prefill(cuda_lib, c, q, counts, 4), q, counts, 0.125, 0, 0, weights_16bit=True)
    assert status(cuda_lib) == GDN_OK
