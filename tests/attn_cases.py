"""Plain forms of the attention layer's calls, in 64 bits on the host, and the inputs of their
tests.

Bound of the attention outputs. With w_j the weights, o = sum w_j v_j / sum w_j:
  - a score s = scale q.k summed in fp32 over D terms is off by about
    4 sqrt(D) 2^-24 scale |q| |k| (rounding errors of D terms add up like a random walk;
    four of its standard deviations), and a relative error e of every weight moves o by at
    most 2 e max|v|;
  - the exponential, its argument's product and the sums of weights add 2^-20;
  - weights held in a 16-bit type (the prompt form) add half a unit of that type, u max|v|;
  - the output is rounded once: u |o|.
"""
import numpy as np

UNIT = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def bound(ref, q, k, v, scale, dtype, weights_16bit=False):
    d = q.shape[-1]
    reach = abs(scale) * np.sqrt((q ** 2).sum(-1).max() * (k ** 2).sum(-1).max())
    vmax = np.abs(v).max()
    e = 4 * np.sqrt(d) * 2.0 ** -24 * reach + 2.0 ** -20
    if weights_16bit and dtype != "float32":
        e += UNIT[dtype] / 2
    return UNIT[dtype] * np.abs(ref) + 2 * e * vmax


def attention(q, k, v, first, scale, window, sinks):
    """q [m][Hq][D] at positions first .., k, v [L][Hkv][D]; 64-bit numpy."""
    m, hq, _ = q.shape
    n, hkv, _ = k.shape
    out = np.zeros(q.shape)
    j = np.arange(n)
    for t in range(m):
        p = first + t
        see = (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))
        if not see.any():
            continue
        for h in range(hq):
            kv = h // (hq // hkv)
            s = scale * (k[see, kv] @ q[t, h])
            w = np.exp(s - s.max())
            out[t, h] = (w @ v[see, kv]) / w.sum()
    return out


class Cache:
    """A paged cache holding sequences of given lengths, its pages in a shuffled order, every
    byte that no position owns a NaN."""

    def __init__(self, torch, rng, lens, hkv, d, ps, dtype, pool=None, spare_cols=1,
                 evicted=None):
        self.torch, self.lens, self.ps = torch, list(lens), ps
        self.hkv, self.d, self.dtype = hkv, d, dtype
        self.pool = pool or len(lens)
        self.slots = rng.permutation(self.pool)[:len(lens)]
        need = [-(-n // ps) for n in lens]
        self.n_pages = sum(need) + 3
        self.max_pages = max(need + [1]) + spare_cols
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.pool, self.max_pages), -1, np.int32)
        self.kv_lens = np.zeros(self.pool, np.int32)
        self.k = [rng.standard_normal((n, hkv, d)) for n in lens]
        self.v = [rng.standard_normal((n, hkv, d)) for n in lens]
        kp = np.full((self.n_pages, hkv, ps, d), np.nan)
        vp = kp.copy()
        at = 0
        for i, n in enumerate(lens):
            row = ids[at:at + need[i]]
            at += need[i]
            self.table[self.slots[i], :need[i]] = row
            self.kv_lens[self.slots[i]] = n
            self.k[i] = self.typed(self.k[i])
            self.v[i] = self.typed(self.v[i])
            for c, page in enumerate(row):
                part = slice(c * ps, min(n, (c + 1) * ps))
                m = part.stop - part.start
                kp[page, :, :m] = self.k[i][part].transpose(1, 0, 2)
                vp[page, :, :m] = self.v[i][part].transpose(1, 0, 2)
        # pages of keys that nobody sees any more are gone: their ids point nowhere
        for i, (lo, hi) in enumerate(evicted or []):
            for c in range(-(-lo // ps), hi // ps):
                self.table[self.slots[i], c] = 1 << 30
        self.k_pages, self.v_pages = self.dev(kp), self.dev(vp)
        ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        self.d_table, self.d_lens, self.d_slots = ints(self.table), ints(self.kv_lens), ints(self.slots)

    def typed(self, x):
        """x rounded to the cache's type, as 64-bit numpy."""
        return self.torch.from_numpy(x).to(getattr(self.torch, self.dtype)).double().numpy()

    def dev(self, x):
        return self.torch.from_numpy(np.ascontiguousarray(x)).to(getattr(self.torch, self.dtype)).cuda()

    def sizes(self):
        return dict(page_size=self.ps, n_pages=self.n_pages, max_pages=self.max_pages)

    def queries(self, rng, counts, hq):
        """Queries of the last counts[i] positions of every sequence: packed [rows][Hq][D]."""
        return self.typed(2 * rng.standard_normal((sum(counts), hq, self.d)))

    def check(self, out, q, counts, scale, window, sinks, weights_16bit=False):
        """Every output row against the 64-bit form."""
        got = out.double().cpu().numpy().reshape(q.shape)
        at = 0
        for i, m in enumerate(counts):
            if m == 0:
                continue
            ref = attention(q[at:at + m], self.k[i], self.v[i], self.lens[i] - m, scale, window, sinks)
            err = np.abs(got[at:at + m] - ref)
            assert np.isfinite(got[at:at + m]).all(), f"sequence {i}: values that are not finite"
            if self.lens[i]:
                tol = bound(ref, q[at:at + m], self.k[i], self.v[i], scale, self.dtype, weights_16bit)
                assert (err <= tol).all(), f"sequence {i}: off by {(err / tol).max():.2f} of the bound"
            else:
                assert (got[at:at + m] == 0).all(), f"sequence {i} sees nothing and is not zero"
            at += m
