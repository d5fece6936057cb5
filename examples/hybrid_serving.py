"""A small hybrid model served from one pool of slots: Gated-DeltaNet blocks and attention
layers (one with a sliding window and sinks, one that sees everything) over a shared paged
cache, with random weights.

    python examples/hybrid_serving.py

A batch of prompts is read in, every sequence is forked into a second continuation, single
tokens are decoded, drafts are verified and what the model did not agree with is rolled
back (recurrent states by snapshot, cache by truncation), half of the sequences are
released and the pages of the others moved together. Tokens, lengths and tables stay on the
device; torch multiplies the projections and holds the memory.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_scan_gb300 as gdn  # noqa: E402

EPS = 1e-6


def rms_norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


class RecurrentLayer:
    """A Gated-DeltaNet block with its projections and the states of every slot."""

    def __init__(self, width, n_slots, n_k_heads=2, n_v_heads=4, state_size=64, conv_kernel=4):
        self.hk, self.h, self.s, self.kernel = n_k_heads, n_v_heads, state_size, conv_kernel
        self.conv_dim = (2 * n_k_heads + n_v_heads) * state_size
        inner = n_v_heads * state_size
        self.w = {name: torch.randn(width, cols, device="cuda") / math.sqrt(width)
                  for name, cols in (("qkv", self.conv_dim), ("alpha", n_v_heads),
                                     ("b", n_v_heads), ("z", inner))}
        self.w_out = torch.randn(inner, width, device="cuda") / math.sqrt(inner)
        self.conv_w = 0.5 * torch.randn(self.conv_dim, conv_kernel, device="cuda")
        self.dt = 0.5 * torch.randn(n_v_heads, device="cuda")
        self.a = -torch.exp(torch.rand(n_v_heads, device="cuda") - 0.5)
        self.norm_w = torch.ones(state_size, device="cuda")
        self.state = torch.zeros(n_slots, n_v_heads, state_size, state_size, device="cuda")
        self.conv = torch.zeros(n_slots, self.conv_dim, conv_kernel - 1, device="cuda")

    def _inputs(self, x):
        p = {name: x @ w for name, w in self.w.items()}
        return (p["qkv"], self.conv_w, self.conv, p["alpha"], p["b"], self.dt, self.a, p["z"],
                self.norm_w, self.state)

    def _sizes(self):
        return (self.hk, self.h, self.s, self.kernel, 1 / math.sqrt(self.s), EPS, EPS)

    def forward(self, x, batch):
        out = x.new_empty(x.shape[0], self.h, self.s)
        common = dict(slots=batch.slots, pool=self.state.shape[0], err_count=batch.errors)
        if batch.cu is not None:
            work = x.new_empty(gdn.gdn_block_prefill_varlen_workspace_size(
                batch.n, x.shape[0], self.hk, self.h, self.s) // 4 + 1)
            gdn.gdn_block_prefill_varlen(*self._inputs(x), out, batch.cu, batch.n, x.shape[0],
                                         batch.longest, *self._sizes(), work, **common)
        elif batch.tokens == 1:
            gdn.gdn_block_decode(*self._inputs(x), out, batch.n, *self._sizes(), **common)
        else:
            self.snaps = x.new_empty(x.shape[0], *self.state.shape[1:])
            self.conv_snaps = x.new_empty(x.shape[0], *self.conv.shape[1:])
            work = x.new_empty(gdn.gdn_block_prefill_workspace_size(
                batch.n, batch.tokens, self.hk, self.h, self.s) // 4 + 1)
            gdn.gdn_block_prefill_snapshots(*self._inputs(x), out, self.snaps, self.conv_snaps,
                                            batch.n, batch.tokens, *self._sizes(), work, **common)
        return out.flatten(1) @ self.w_out

    def roll_back(self, batch, accepted):
        """Every sequence of a verified batch to the state after its accepted tokens."""
        gdn.gdn_snapshot_restore(self.state, self.snaps, accepted, batch.n, batch.tokens, self.h,
                                 self.s, self.conv, self.conv_snaps, self.conv_dim, self.kernel,
                                 slots=batch.slots, pool=self.state.shape[0],
                                 err_count=batch.errors)

    def copy_slots(self, parents, children):
        self.state[children.long()] = self.state[parents.long()]
        self.conv[children.long()] = self.conv[parents.long()]

    def clear_slots(self, slots):
        self.state[slots.long()] = 0
        self.conv[slots.long()] = 0


class AttentionLayer:
    """An attention layer: one projection to q, k and v, whose slices the calls take as they
    lie, and the layer's two planes of the paged cache."""

    def __init__(self, width, cache, layer, n_q_heads, window=0, n_sinks=0):
        self.cache, self.layer, self.hq = cache, layer, n_q_heads
        self.window, self.sinks = window, n_sinks
        d, hkv = cache.head_dim, cache.n_kv_heads
        self.w_qkv = torch.randn(width, (n_q_heads + 2 * hkv) * d, device="cuda") / math.sqrt(width)
        self.w_out = torch.randn(n_q_heads * d, width, device="cuda") / math.sqrt(n_q_heads * d)

    def forward(self, x, batch):
        c, hkv, d = self.cache, self.cache.n_kv_heads, self.cache.head_dim
        rows = (x @ self.w_qkv).to(c.dtype).view(x.shape[0], self.hq + 2 * hkv, d)
        q, k, v = rows.split((self.hq, hkv, hkv), dim=1)
        k_pages, v_pages = c.planes[2 * self.layer], c.planes[2 * self.layer + 1]
        books = (k_pages, v_pages, c.table, c.lens)
        pages = (c.page_size, c.n_pages, c.max_pages)
        common = dict(slots=batch.slots, pool=c.pool, err_count=batch.errors)
        gdn.gdn_kv_append(k, v, *books, batch.cu, batch.n, x.shape[0], hkv, d, *pages, **common)
        out = torch.empty(x.shape[0], self.hq, d, device="cuda", dtype=c.dtype)
        mask = (self.window, self.sinks, 1 / math.sqrt(d))
        if batch.cu is not None:
            gdn.gdn_attn_prefill(q, *books, out, batch.cu, batch.n, x.shape[0], batch.longest,
                                 self.hq, hkv, d, *pages, *mask, **common)
        else:
            work = torch.empty(gdn.gdn_attn_decode_workspace_size(
                batch.n, batch.tokens, self.hq, hkv, d), device="cuda", dtype=torch.uint8)
            gdn.gdn_attn_decode(q, *books, out, batch.n, batch.tokens, self.hq, hkv, d, *pages,
                                *mask, work, **common)
        return out.flatten(1).float() @ self.w_out


class Cache:
    """The pages of every attention layer, and the books that say whose they are."""

    def __init__(self, n_layers, pool, n_pages, max_pages, n_kv_heads, page_size, head_dim, dtype):
        self.pool, self.n_pages, self.max_pages = pool, n_pages, max_pages
        self.n_kv_heads, self.page_size, self.head_dim, self.dtype = (n_kv_heads, page_size,
                                                                      head_dim, dtype)
        self.planes = torch.empty(2 * n_layers, n_pages, n_kv_heads, page_size, head_dim,
                                  device="cuda", dtype=dtype)
        ints = dict(device="cuda", dtype=torch.int32)
        self.table = torch.full((pool, max_pages), -1, **ints)
        self.lens = torch.zeros(pool, **ints)
        self.refs = torch.zeros(n_pages, **ints)
        self.live = torch.zeros(1, **ints)
        self.work = torch.empty(gdn.gdn_pages_workspace_size(pool, n_pages), device="cuda",
                                dtype=torch.uint8)
        page_bytes = n_kv_heads * page_size * head_dim * self.planes.element_size()
        self._data = (2 * n_layers, n_pages, page_bytes, max_pages)

    def reserve(self, slots, n_new, errors):
        gdn.gdn_pages_reserve(self.planes, self.table, self.lens, self.refs, n_new, slots.numel(),
                              self.page_size, *self._data, self.work, slots=slots, pool=self.pool,
                              err_count=errors)

    def fork(self, parents, children, errors):
        gdn.gdn_pages_fork(self.planes, self.table, self.lens, self.refs, parents, children,
                           parents.numel(), self.page_size, *self._data, self.pool, self.work,
                           err_count=errors)

    def truncate(self, slots, new_lens, errors):
        gdn.gdn_pages_truncate(self.table, self.lens, self.refs, new_lens, slots.numel(),
                               self.page_size, self.n_pages, self.max_pages, slots=slots,
                               pool=self.pool, err_count=errors)

    def compact(self):
        gdn.gdn_pages_compact(self.planes, self.table, self.lens, self.refs, self.page_size,
                              *self._data, self.pool, self.work, n_live=self.live)


class Batch:
    """What one step runs on: the slots, and the rows each of them has (ragged, or the same
    number for all)."""

    def __init__(self, slots, errors, lengths=None, tokens=0):
        self.slots, self.errors, self.n, self.tokens = slots, errors, slots.numel(), tokens
        self.cu, self.longest = None, tokens
        if lengths is not None:
            self.longest = max(lengths)
            ends = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0, dtype=torch.int32)
            self.cu = ends.cuda()
            self.n_new = torch.tensor(lengths, device="cuda", dtype=torch.int32)
        else:
            self.n_new = torch.full((self.n,), tokens, device="cuda", dtype=torch.int32)


class Server:
    def __init__(self, width=256, vocab=512, pool=32, n_pages=256, max_pages=32, page_size=16,
                 n_q_heads=8, n_kv_heads=2, head_dim=64, window=64, n_sinks=4,
                 dtype=torch.float32, seed=0):
        torch.manual_seed(seed)
        self.cache = Cache(2, pool, n_pages, max_pages, n_kv_heads, page_size, head_dim, dtype)
        self.layers = [RecurrentLayer(width, pool),
                       AttentionLayer(width, self.cache, 0, n_q_heads, window, n_sinks),
                       RecurrentLayer(width, pool),
                       AttentionLayer(width, self.cache, 1, n_q_heads)]
        self.embedding = torch.randn(vocab, width, device="cuda")
        self.errors = torch.zeros(1, device="cuda", dtype=torch.int32)

    def _run(self, batch, tokens):
        """The logits of every row of a batch whose pages are reserved."""
        x = self.embedding[tokens]
        for layer in self.layers:
            x = x + layer.forward(rms_norm(x), batch)
        return rms_norm(x) @ self.embedding.T / math.sqrt(x.shape[1])

    def _step(self, batch, tokens):
        self.cache.reserve(batch.slots, batch.n_new, self.errors)
        return self._run(batch, tokens)

    def prompt(self, slots, tokens, lengths):
        """Logits of every token of the packed prompts, which continue what the slots hold."""
        return self._step(Batch(slots, self.errors, lengths=lengths), tokens)

    def decode(self, slots, tokens):
        """One more token of every slot: [n] -> logits [n][vocab]."""
        return self._step(Batch(slots, self.errors, tokens=1), tokens)

    def verify(self, slots, tokens):
        """Tokens [n][m], the first of them certain, the others drafts: keeps the drafts the
        model agrees with. Returns (logits [n][m][vocab], how many of the m were kept)."""
        n, m = tokens.shape
        batch = Batch(slots, self.errors, tokens=m)
        logits = self._step(batch, tokens.flatten()).view(n, m, -1)
        agree = (logits.argmax(-1)[:, :-1] == tokens[:, 1:]).int().cumprod(1)
        kept = 1 + agree.sum(1, dtype=torch.int32)
        for layer in self.layers:
            if isinstance(layer, RecurrentLayer):
                layer.roll_back(batch, kept)
        self.cache.truncate(slots, self.cache.lens[slots.long()] - m + kept, self.errors)
        return logits, kept

    def fork(self, parents, children):
        self.cache.fork(parents, children, self.errors)
        for layer in self.layers:
            if isinstance(layer, RecurrentLayer):
                layer.copy_slots(parents, children)

    def release(self, slots):
        self.cache.truncate(slots, None, self.errors)
        for layer in self.layers:
            if isinstance(layer, RecurrentLayer):
                layer.clear_slots(slots)

    def check(self):
        """Waits for the device; raises if a call skipped anything or gave up a wait."""
        gdn.gdn_device_error()
        if self.errors.item():
            raise RuntimeError(f"{self.errors.item()} sequences, rows or pages were skipped")


def main():
    torch.cuda.set_device(0)
    server = Server(dtype=torch.bfloat16)
    ints = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    lengths = [1, 150, 37, 64]
    slots, twins = ints(3, 0, 9, 17), ints(4, 1, 10, 18)
    logits = server.prompt(slots, torch.randint(512, (sum(lengths),), device="cuda"), lengths)
    last = torch.tensor(lengths, device="cuda").cumsum(0) - 1
    server.fork(slots, twins)
    everyone = torch.cat([slots, twins])
    best = logits[last].topk(2).indices
    tokens = best.T.flatten()           # the twin of a sequence goes on with the second choice
    for _ in range(20):
        tokens = server.decode(everyone, tokens).argmax(-1)
    drafts = torch.cat([tokens[:, None], torch.randint(512, (8, 3), device="cuda")], 1)
    _, kept = server.verify(everyone, drafts)
    print("drafts kept, the certain token among them:", kept.tolist())
    server.release(slots)
    server.cache.compact()
    server.check()
    print("lengths:", server.cache.lens[twins.long()].tolist(),
          "pages in use:", server.cache.live.item(), "of", server.cache.n_pages)


if __name__ == "__main__":
    main()
