"""What the attention kernels do once a bounded wait gave up.

A copy of the kernels (tests/cuda/give_up_*.cu: their own sources, with one wait that returns
at once as if it had run out, and the others bounded by 50 ms) runs with the give-up at chosen
waits of every kind of warp, in all of its lanes or in one of them only. The call has to end,
to raise its flag, to write nothing but right rows, and to leave the next call unharmed. No
wait is without a bound, nothing faults, and what was in flight has landed when a CTA leaves."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests.attn_cases import Cache, attention, bound
from tests.test_attn_decode_gpu import run as decode
from tests.test_attn_prefill_gpu import run as prefill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_linear_scan_gb300", "csrc")


class Copy:
    """The binding with the library replaced by the copy (which has the attention call only)."""

    def __init__(self, gdn, lib, monkeypatch, names):
        self.gdn, self.lib = gdn, lib
        for name in names:
            getattr(lib, name).argtypes, getattr(lib, name).restype = gdn._SIGS[name]
        lib.give_up_flags.restype = ctypes.c_uint
        monkeypatch.setattr(gdn, "library", lambda: lib)

    def arm(self, cta, warp, nth, lanes):
        torch.cuda.synchronize()
        assert self.lib.give_up_arm(cta, warp, nth, ctypes.c_uint(lanes)) == 0

    def ended(self):
        """(whether a wait gave up, the waits of the armed warp) once the call has ended."""
        torch.cuda.synchronize()
        return self.lib.give_up_flags() != 0, self.lib.give_up_waits()


def build(name, where):
    out = str(where / f"lib{name}.so")
    subprocess.run(["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                    "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, "-I",
                    os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "cuda", f"{name}.cu"),
                    "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.fixture(scope="module")
def prompt_lib(tmp_path_factory):
    return build("give_up_prompt", tmp_path_factory.mktemp("prompt"))


@pytest.fixture(scope="module")
def decode_lib(tmp_path_factory):
    return build("give_up_decode", tmp_path_factory.mktemp("decode"))


class Wanted:
    """The 64-bit form's rows and the bound of every value."""

    def __init__(self, c, q, counts, scale, weights_16bit):
        refs, tols, at = [], [], 0
        for i, m in enumerate(counts):
            x = q[at:at + m]
            refs.append(attention(x, c.k[i], c.v[i], c.lens[i] - m, scale, 0, 0))
            tols.append(bound(refs[-1], x, c.k[i], c.v[i], scale, c.dtype, weights_16bit))
            at += m
        self.ref, self.tol = np.concatenate(refs), np.concatenate(tols)

    def untouched(self, out):
        """How many rows hold what they held before (NaN); the others have to be right."""
        got = out.double().cpu().numpy().reshape(self.ref.shape)
        old = np.isnan(got).all(-1)
        assert (old[..., None] | (np.abs(got - self.ref) <= self.tol)).all(), "a wrong row"
        return int(old.sum())


# warps of a CTA: eight (head_dim 256: four) of softmax, then MMA, K, V, scheduling
@pytest.mark.parametrize("d,dtype", [(64, "float16"), (128, "bfloat16"), (256, "bfloat16")])
def test_prompt(cuda_lib, prompt_lib, monkeypatch, d, dtype):
    """More pairs of row tiles than CTAs at a time, so that a CTA takes several."""
    rng = np.random.default_rng(d)
    counts = [300, 129] + [1 + i % 20 for i in range(90)]
    lens = [m + 17 * (i % 9) for i, m in enumerate(counts)]
    scale = d ** -0.5
    c = Cache(torch, rng, lens, 5, d, 16, dtype)
    q = c.queries(rng, counts, 10)
    wanted = Wanted(c, q, counts, scale, True)
    call = Copy(cuda_lib, prompt_lib, monkeypatch, ["gdn_attn_prefill", "gdn_attn_prefill_workspace_size"])
    softmax = 4 if d == 256 else 8
    for warp in (0, 1, softmax - 1, softmax, softmax + 1, softmax + 2, softmax + 3):
        for nth in (0, 1, 2, 5, 9):
            for lanes in (0xFFFFFFFF, 1 << (5 + 3 * nth) % 32):
                call.arm(3, warp, nth, lanes)
                out = prefill(cuda_lib, c, q, counts, 10)
                flag, waits = call.ended()
                assert flag == (waits > nth) and (flag or nth > 1)
                left = wanted.untouched(out)
                assert flag or left == 0
                # (the scheduling warp's and the second row tile's may come too late to matter)
                assert left > 0 or nth > 0 or warp not in (0, softmax, softmax + 1, softmax + 2)
    call.arm(-1, 0, 0, 0)
    assert wanted.untouched(prefill(cuda_lib, c, q, counts, 10)) == 0
    assert call.ended()[0] is False
    monkeypatch.undo()
    assert wanted.untouched(prefill(cuda_lib, c, q, counts, 10)) == 0
    cuda_lib.gdn_device_error()


DECODE = ["gdn_attn_decode", "gdn_attn_decode_workspace_size"]


# warps of a CTA: four that compute, the loading warp, the joining one (fp32 with heads of 64 and
# few rows has none)
@pytest.mark.parametrize("d,dtype,warps", [(64, "float32", 5), (128, "float16", 6), (64, "bfloat16", 6),
                                           (256, "bfloat16", 6), (128, "float32", 6)])
def test_decode(cuda_lib, decode_lib, monkeypatch, d, dtype, warps):
    """Units that are whole, split in two and split over many CTAs."""
    rng = np.random.default_rng(d)
    lens = [70000] + [int(x) for x in rng.integers(1, 1500, 600)] + [20000]
    n, scale = len(lens), d ** -0.5
    c = Cache(torch, rng, lens, 1, d, 64, dtype)
    q = c.queries(rng, [1] * n, 2)
    wanted = Wanted(c, q, [1] * n, scale, False)
    call = Copy(cuda_lib, decode_lib, monkeypatch, DECODE)
    for cta in (1, 20, 140):
        for warp in range(warps):
            for nth in (0, 1, 4, 11):
                for lanes in (0xFFFFFFFF, 1 << (5 + 3 * nth) % 32):
                    call.arm(cta, warp, nth, lanes)
                    out = decode(cuda_lib, c, q, 1, 2)
                    flag, waits = call.ended()
                    assert flag == (waits > nth) and (flag or nth > 0)
                    left = wanted.untouched(out)
                    assert flag or left == 0
                    # (what the joining warp waits for, and a loading warp at its last tile, may
                    # come too late to matter)
                    assert left > 0 or nth > 0 or warp >= 4
    call.arm(-1, 0, 0, 0)
    assert wanted.untouched(decode(cuda_lib, c, q, 1, 2)) == 0
    assert call.ended()[0] is False
    monkeypatch.undo()
    assert wanted.untouched(decode(cuda_lib, c, q, 1, 2)) == 0
    cuda_lib.gdn_device_error()


@pytest.mark.parametrize("d,dtype,warps", [(64, "float32", 5), (128, "bfloat16", 6), (256, "float16", 6)])
@pytest.mark.parametrize("lens", [[150000], [70000, 900, 20000, 31000]])
def test_replays_after_a_give_up(cuda_lib, decode_lib, monkeypatch, d, dtype, warps, lens):
    """A captured decode call, replayed with and without a wait that gives up: every replay leaves
    the workspace's counts (its first words, one per CTA) cleared, a replay in which a wait gave
    up writes no wrong row, and the next one gives the bits of an undisturbed call."""
    rng = np.random.default_rng([d, len(lens)])
    n, scale, ctas = len(lens), d ** -0.5, 3 * 152
    c = Cache(torch, rng, lens, 1, d, 64, dtype)
    q = c.queries(rng, [1] * n, 2)
    wanted = Wanted(c, q, [1] * n, scale, False)
    clean = decode(cuda_lib, c, q, 1, 2)
    assert wanted.untouched(clean) == 0
    call = Copy(cuda_lib, decode_lib, monkeypatch, DECODE)
    call.arm(-1, 0, 0, 0)
    qd, out = c.dev(q), torch.empty_like(clean)
    ws = torch.zeros(cuda_lib.gdn_attn_decode_workspace_size(n, 1, 2, 1, d), dtype=torch.uint8, device="cuda")
    run = lambda: cuda_lib.gdn_attn_decode(  # noqa: E731
        qd, c.k_pages, c.v_pages, c.d_table, c.d_lens, out, n, 1, 2, 1, d, 64, c.n_pages, c.max_pages,
        0, 0, scale, ws, slots=c.d_slots, pool=c.pool)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for cta in (0, 1, 77, 151):
        for warp in range(warps):
            for nth in (0, 2, 5):
                call.arm(cta, warp, nth, 0xFFFFFFFF if nth else 1 << (3 * warp + 1))
                out.fill_(float("nan"))
                graph.replay()
                flag, waits = call.ended()
                assert flag == (waits > nth)
                left = wanted.untouched(out)
                assert flag or left == 0
                where = f"after CTA {cta}, warp {warp}, wait {nth}"
                assert not ws[:8 * ctas].any(), f"counts left {where}"
                call.arm(-1, 0, 0, 0)
                out.fill_(float("nan"))
                graph.replay()
                assert call.ended()[0] is False
                assert torch.equal(out, clean), f"other bits {where}"
                assert not ws[:8 * ctas].any()
