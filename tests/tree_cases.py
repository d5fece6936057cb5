"""Trees of drafted tokens for the tests, and plain forms in 64 bits of the calls on them.

Bound of the block's outputs. SiLU is good to 1e-5 relative where the conv output is not far below
zero (documented), so q, k and v are, and with them u (|u| <= |v| + |S0 k| a step, the delta rule's
matrix I - beta k k^T does not lengthen) and y. The gated norm divides y by its own size, and
multiplies by another SiLU: relative errors stay, absolute ones are those of y over its RMS. So an
output of size 1 is off by a few 1e-5: the framework's bound of one step, 1e-4 + 1e-4 |ref|, holds for
every node of a tree too, with the head's largest output as the size where y's elements differ."""
import numpy as np

NO_NODE = -2


def random_tree(rng, n_nodes, there=None, chain=0.4, roots=1):
    """Parents of a tree of `there` nodes (padded to n_nodes): a node hangs from the one before it
    with probability `chain`, else from any; the first `roots` are roots."""
    m = n_nodes if there is None else there
    out = [-1 if i < roots else i - 1 if rng.random() < chain else int(rng.integers(i)) for i in range(m)]
    return out + [NO_NODE] * (n_nodes - m)


def valid(tree):
    """(which nodes are there, whether some parent is not valid)."""
    there, bad = [], False
    for i, p in enumerate(tree):
        ok = p == -1 or (0 <= p < i and there[p])
        there.append(ok)
        bad = bad or (not ok and p != NO_NODE)
    return there, bad


def path_to(tree, i):
    out = []
    while i >= 0:
        out.append(i)
        i = tree[i]
    return out[::-1]


def attention(q, k, v, tree, scale, window, sinks):
    """q [N][Hq][D] of the nodes, k, v [L][Hkv][D] of the whole cache (the last N rows the nodes')."""
    n, hq, _ = q.shape
    length, hkv, _ = k.shape
    base = length - n
    there, _ = valid(tree)
    depth = [len(path_to(tree, i)) - 1 if there[i] else 0 for i in range(n)]
    out = np.zeros(q.shape)
    for i in range(n):
        if not there[i]:
            continue
        p = base + depth[i]
        rows, at = list(range(base)), list(range(base))
        for a in path_to(tree, i):
            rows.append(base + a)
            at.append(base + depth[a])
        rows, at = np.array(rows), np.array(at)
        see = (window == 0) | (p - at < window) | (at < sinks)
        rows = rows[see]
        for h in range(hq):
            kv = h // (hq // hkv)
            s = scale * (k[rows, kv] @ q[i, h])
            w = np.exp(s - s.max())
            out[i, h] = (w @ v[rows, kv]) / w.sum()
    return out


def _silu(x):
    return x / (1 + np.exp(-x))


class Block:
    """Inputs of a block over trees, and its plain form."""

    def __init__(self, rng, trees, hk, h, s, kernel, pool=None, slots=None, decay=2.0):
        n, t = len(trees), len(trees[0])
        self.trees, self.n, self.t = trees, n, t
        self.hk, self.h, self.s, self.kernel = hk, h, s, kernel
        self.pool = pool or n
        self.slots = list(range(n)) if slots is None else slots
        c = (2 * hk + h) * s
        f = lambda *shape: rng.standard_normal(shape).astype(np.float32)  # noqa: E731
        self.qkv, self.conv_w, self.z = f(n, t, c), 0.5 * f(c, kernel), f(n, t, h, s)
        self.conv_state, self.state = f(self.pool, c, kernel - 1), 0.1 * f(self.pool, h, s, s)
        self.a, self.dt = -np.exp(0.5 * f(h)), 0.5 * f(h)
        g = -rng.uniform(0.001, decay, (n, t, h))
        self.alpha = (np.log(np.expm1(g / self.a)) - self.dt).astype(np.float32)
        self.b, self.norm_w = f(n, t, h), (1 + 0.1 * f(s)).astype(np.float32)
        self.scale, self.eps = 1 / np.sqrt(s), 1e-6
        # what a node that is not there holds must not matter
        for x, tree in enumerate(trees):
            there, _ = valid(tree)
            for i in range(t):
                if not there[i]:
                    for arr in (self.qkv, self.alpha, self.b, self.z):
                        arr[x, i] = np.nan

    def step(self, x, i, state, hist):
        """(state, history, output) behind node i of sequence x, from its parent's."""
        hk, h, s = self.hk, self.h, self.s
        d = lambda v: v.astype(np.float64)  # noqa: E731
        taps = np.concatenate([hist, d(self.qkv[x, i])[:, None]], 1)
        y = _silu((taps * d(self.conv_w)).sum(1))
        unit = lambda v: v / np.maximum(np.linalg.norm(v, axis=-1, keepdims=True), self.eps)  # noqa: E731
        q, k = unit(y[:hk * s].reshape(hk, s)), unit(y[hk * s:2 * hk * s].reshape(hk, s))
        v = y[2 * hk * s:].reshape(h, s)
        g = self.a * np.logaddexp(0, d(self.alpha[x, i]) + self.dt)
        beta = 1 / (1 + np.exp(-d(self.b[x, i])))
        heads = np.arange(h) % hk
        state = state * np.exp(g)[:, None, None]
        delta = (v - np.einsum("hji,hi->hj", state, k[heads])) * beta[:, None]
        state = state + np.einsum("hj,hi->hji", delta, k[heads])
        o = self.scale * np.einsum("hji,hi->hj", state, q[heads])
        o = o / np.sqrt((o * o).mean(-1, keepdims=True) + self.eps) * self.norm_w * _silu(d(self.z[x, i]))
        return state, taps[:, 1:], o

    def run(self, x):
        """(outputs [t][h][s], states and histories behind every node) of sequence x."""
        slot, tree = self.slots[x], self.trees[x]
        there, _ = valid(tree)
        out, after = np.zeros((self.t, self.h, self.s)), {}
        after[-1] = (self.state[slot].astype(np.float64), self.conv_state[slot].astype(np.float64))
        for i, p in enumerate(tree):
            if there[i]:
                state, hist, out[i] = self.step(x, i, *after[p])
                after[i] = (state, hist)
        return out, after
