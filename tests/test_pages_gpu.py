"""The paged cache's bookkeeping against a plain model of it on the host: the same tables,
lengths and reference counts, and the same bytes in every page."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Model:
    """The books and pages in plain Python; one method per call, in the order of the call."""

    def __init__(self, rng, n_slots, n_pages, ps, max_pages, planes=3, page_bytes=48):
        self.ps, self.n_pages, self.max_pages, self.planes = ps, n_pages, max_pages, planes
        self.page_bytes, self.pool = page_bytes, n_slots
        self.table = np.full((n_slots, max_pages), -1, np.int32)
        self.lens = np.zeros(n_slots, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.pages = rng.integers(0, 256, (planes, n_pages, page_bytes)).astype(np.uint8)
        self.errors = 0

    def cols(self, n):
        return -(-int(n) // self.ps)

    def free(self):
        return [int(p) for p in np.nonzero(self.refs == 0)[0]]

    def reserve(self, slots, add):
        free, used, before = self.free(), 0, self.refs.copy()
        for s, a in zip(slots, add):
            n = int(self.lens[s]) if 0 <= s < self.pool else -1
            if n < 0 or a < 0 or n + a > self.max_pages * self.ps:
                self.errors += 1
                continue
            cow = a > 0 and n % self.ps and before[self.table[s, n // self.ps]] > 1
            need = self.cols(n + a) - self.cols(n) + bool(cow)
            mine = free[used:used + need]
            used += need
            if used > len(free):
                self.errors += 1
                continue
            if cow:
                old, new = self.table[s, n // self.ps], mine.pop(0)
                self.pages[:, new] = self.pages[:, old]
                self.table[s, n // self.ps] = new
                self.refs[old] -= 1
                self.refs[new] = 1
            for c in range(self.cols(n), self.cols(n + a)):
                self.table[s, c] = mine.pop(0)
                self.refs[self.table[s, c]] = 1
            self.lens[s] = n + a

    def fork(self, parents, children):
        free, used = self.free(), 0
        lens = self.lens.copy()
        for a, b in zip(parents, children):
            if not (0 <= a < self.pool and 0 <= b < self.pool) or lens[b] != 0 or a == b:
                self.errors += 1
                continue
            n = int(lens[a])
            if n % self.ps:
                used += 1
                if used > len(free):
                    self.errors += 1
                    continue
            full = n // self.ps
            self.table[b, :full] = self.table[a, :full]
            for p in self.table[a, :full]:
                self.refs[p] += 1
            if n % self.ps:
                new, old = free[used - 1], self.table[a, full]
                self.pages[:, new] = self.pages[:, old]
                self.table[b, full] = new
                self.refs[new] = 1
            self.lens[b] = n

    def truncate(self, slots, keep):
        for s, k in zip(slots, keep):
            if not 0 <= s < self.pool or not 0 <= k <= self.lens[s]:
                self.errors += 1
                continue
            for c in range(self.cols(k), self.cols(self.lens[s])):
                self.refs[self.table[s, c]] -= 1
                self.table[s, c] = -1
            self.lens[s] = k

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, self.n_pages) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        for a, b in zip(src, dst):
            self.pages[:, b] = self.pages[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return live


class Device:
    """The same books on the GPU, through the library."""

    def __init__(self, gdn, m):
        self.gdn, self.m = gdn, m
        up = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
        self.table, self.lens, self.refs, self.pages = up(m.table), up(m.lens), up(m.refs), up(m.pages)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.data = (m.ps, m.planes, m.n_pages, m.page_bytes, m.max_pages)

    def ws(self, n):
        size = self.gdn.gdn_pages_workspace_size(n, self.m.n_pages)
        return torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")

    @staticmethod
    def ints(x):
        return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")

    def reserve(self, slots, add):
        self.gdn.gdn_pages_reserve(self.pages, self.table, self.lens, self.refs, self.ints(add),
                                   len(slots), *self.data, self.ws(len(slots)),
                                   slots=self.ints(slots), pool=self.m.pool, err_count=self.err)

    def fork(self, parents, children):
        self.gdn.gdn_pages_fork(self.pages, self.table, self.lens, self.refs, self.ints(parents),
                                self.ints(children), len(parents), *self.data, self.m.pool,
                                self.ws(len(parents)), err_count=self.err)

    def truncate(self, slots, keep):
        self.gdn.gdn_pages_truncate(self.table, self.lens, self.refs,
                                    None if keep is None else self.ints(keep), len(slots),
                                    self.m.ps, self.m.n_pages, self.m.max_pages,
                                    slots=self.ints(slots), pool=self.m.pool, err_count=self.err)

    def compact(self):
        live = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        self.gdn.gdn_pages_compact(self.pages, self.table, self.lens, self.refs, *self.data,
                                   self.m.pool, self.ws(0), n_live=live)
        return live.item()

    def same(self, what):
        m = self.m
        for name, got, want in (("table", self.table, m.table), ("lengths", self.lens, m.lens),
                                ("references", self.refs, m.refs), ("pages", self.pages, m.pages)):
            assert np.array_equal(got.cpu().numpy(), want), f"{what}: {name} differ"
        assert self.err.item() == m.errors, f"{what}: errors"


@pytest.mark.parametrize("ps,n_slots,n_pages,max_pages", [
    (8, 5, 40, 9), (16, 70, 900, 33), (64, 12, 30, 6), (8, 1500, 9000, 20), (256, 3, 4, 3)])
def test_random_histories(cuda_lib, ps, n_slots, n_pages, max_pages):
    """Reserve, fork, truncate and compact in a random order, running out of pages at times."""
    rng = np.random.default_rng([ps, n_slots])
    m = Model(rng, n_slots, n_pages, ps, max_pages)
    d = Device(cuda_lib, m)
    for step in range(24):
        n = int(rng.integers(1, n_slots + 1))
        slots = rng.permutation(n_slots)[:n]
        kind = step % 4 if step < 8 else int(rng.integers(0, 4))
        if kind == 0:
            add = rng.integers(0, 3 * ps, n) * (rng.random(n) < 0.7)
            m.reserve(slots, add)
            d.reserve(slots, add)
        elif kind == 1:
            empty = np.nonzero(m.lens == 0)[0]
            held = np.nonzero(m.lens > 0)[0]
            if len(empty) == 0 or len(held) == 0:
                continue
            children = rng.permutation(empty)[:n]
            parents = rng.choice(held, len(children))
            m.fork(parents, children)
            d.fork(parents, children)
        elif kind == 2:
            keep = (m.lens[slots] * rng.random(n)).astype(int) * (rng.random(n) < 0.6)
            m.truncate(slots, keep)
            d.truncate(slots, keep)
        else:
            assert m.compact() == d.compact()
        d.same(f"step {step}, kind {kind}")
    every = np.arange(n_slots)
    m.truncate(every, np.zeros(n_slots, int))
    d.truncate(every, None)
    d.same("freed")
    assert not m.refs.any()


def test_out_of_range_is_skipped_and_counted(cuda_lib):
    rng = np.random.default_rng(3)
    m = Model(rng, 6, 20, 8, 4)
    d = Device(cuda_lib, m)
    for slots, add in (([0, 1, 2], [20, 9, 32]), ([6, -1, 0, 1], [1, 1, 13, -1]), ([2], [1])):
        m.reserve(slots, add)
        d.reserve(slots, add)
        d.same("reserve")
    for parents, children in (([0, 0, 6, 1], [0, 1, 3, 9]), ([0, 1], [3, 4])):
        m.fork(parents, children)
        d.fork(parents, children)
        d.same("fork")
    m.truncate([0, 9, 1, 2], [21, 0, -1, 8])
    d.truncate([0, 9, 1, 2], [21, 0, -1, 8])
    d.same("truncate")


def test_a_shared_page_is_copied_before_it_is_written(cuda_lib):
    """Truncated into a page that a fork shares, a sequence gets its own copy as it grows."""
    rng = np.random.default_rng(4)
    m = Model(rng, 4, 16, 8, 5)
    d = Device(cuda_lib, m)
    for side in (m, d):
        side.reserve([0], [16])
        side.fork([0, 0], [1, 2])
        side.truncate([1, 2], [12, 16])
        side.reserve([1, 2], [1, 1])
    d.same("copy on write")
    assert m.table[1, 1] != m.table[0, 1] and m.table[2, 1] == m.table[0, 1]
    assert m.refs[m.table[0, 1]] == 2


@pytest.mark.parametrize("page_bytes,planes", [(16, 1), (4096, 2), (40000, 3)])
def test_copies(cuda_lib, page_bytes, planes):
    rng = np.random.default_rng(page_bytes)
    n_pages = 37
    pages = rng.integers(0, 256, (planes, n_pages, page_bytes)).astype(np.uint8)
    ids = rng.permutation(n_pages).astype(np.int32)
    src, dst = ids[:15].copy(), ids[15:30].copy()
    want = pages.copy()
    want[:, dst] = want[:, src]
    src, dst = np.append(src, [n_pages, 0]), np.append(dst, [1, -1])
    got = torch.from_numpy(pages).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.gdn_pages_copy(got, Device.ints(src), Device.ints(dst), 17, planes, n_pages, page_bytes,
                            err_count=err)
    assert np.array_equal(got.cpu().numpy(), want) and err.item() == 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hkv,d,ps", [(1, 64, 8), (3, 128, 16), (2, 256, 64), (16, 128, 256)])
@pytest.mark.parametrize("uniform,wide", [(False, False), (True, False), (False, True)])
def test_append(cuda_lib, dtype, hkv, d, ps, uniform, wide):
    """Rows land in their pages and nothing else changes."""
    rng = np.random.default_rng([hkv, d, ps])
    new = [2] * 5 if uniform else [1, 0, 37, 2, 300]
    lens = [n + int(rng.integers(0, 90)) for n in new]
    pool, need = 9, [-(-n // ps) for n in lens]
    n_pages, max_pages, total = sum(need) + 2, max(need) + 1, sum(new)
    slots = rng.permutation(pool)[:5]
    table = np.full((pool, max_pages), -1, np.int32)
    ids, at = rng.permutation(n_pages), 0
    for s, m in zip(slots, need):
        table[s, :m] = ids[at:at + m]
        at += m
    kv_lens = np.zeros(pool, np.int32)
    kv_lens[slots] = lens
    shape = (n_pages, hkv, ps, d)
    kp, vp = torch.randn(shape).to(dtype).cuda(), torch.randn(shape).to(dtype).cuda()
    row = torch.randn(total, 3 * hkv, d).to(dtype).cuda()
    k, v = (row[:, hkv:2 * hkv], row[:, 2 * hkv:]) if wide else \
        (row[:, hkv:2 * hkv].contiguous(), row[:, 2 * hkv:].contiguous())
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    want_k, want_v = kp.clone(), vp.clone()
    for i, s in enumerate(slots):
        for t in range(new[i]):
            pos = lens[i] - new[i] + t
            want_k[int(table[s, pos // ps]), :, pos % ps] = k[cu[i] + t]
            want_v[int(table[s, pos // ps]), :, pos % ps] = v[cu[i] + t]
    up = Device.ints
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.gdn_kv_append(k, v, kp, vp, up(table), up(kv_lens), None if uniform else up(cu), 5,
                           total, hkv, d, ps, n_pages, max_pages, slots=up(slots), pool=pool,
                           err_count=err)
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v) and err.item() == 0


def test_append_skips_what_is_out_of_range(cuda_lib):
    """A sequence without room for its rows, a slot and a page out of range: nothing is written
    for them, and each is counted."""
    up = Device.ints
    table, kv_lens = up([[0, 1], [2, 9], [3, 4]]), up([5, 12, 16])
    kp = torch.zeros(5, 1, 8, 64, device="cuda")
    vp = torch.zeros_like(kp)
    k = torch.ones(10, 1, 64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # sequence 0: 6 rows, 5 positions; 1: two rows at 10, 11 in page 9 of 5; 2: slot 7; 3: fine
    cuda_lib.gdn_kv_append(k, k, kp, vp, table, kv_lens, up([0, 6, 8, 9, 10]), 4, 10, 1, 64, 8, 5,
                           2, slots=up([0, 1, 7, 2]), pool=3, err_count=err)
    want = torch.zeros_like(kp)
    want[4, 0, 7] = 1
    assert torch.equal(kp, want) and torch.equal(vp, want) and err.item() == 4
