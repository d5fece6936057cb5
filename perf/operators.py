"""Workloads of the paged attention operators: their inputs, their plain forms, their work.

The attention layers of a hybrid model sit between Gated-DeltaNet blocks and keep their
keys and values in a paged cache: planes of pages [n_pages][n_kv_heads][page_size][head_dim],
a page table and a length per pool slot, and a reference count per page. Four operators:

  append   new tokens' keys and values written to their places in the pages
  decode   attention of one token (or a few draft tokens) of every sequence over its pages
  prompt   attention of a ragged batch of prompts, or chunks of prompts, over their pages
  pages    the bookkeeping: copying, reserving, forking, truncating (freeing), compacting

Attention sees key j from position p when j <= p and (j > p - window, or j < sinks, or
window is 0); query head h reads key head h // (query heads / key heads); a query that
sees nothing gives zeros.

`run` computes in elementary torch operations in 32 bits, or, with `own` set, through the
framework's entry points; `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases

def _attn(name, op, dtype, n, lo, hi, hq, hkv, d, ps, shape, window=0, sinks=0, tokens=1,
          pool=0, empty=0, ctx=0, packed=False):
    return {"name": name, "op": op, "dtype": dtype, "n": n, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "d": d, "ps": ps, "window": window, "sinks": sinks, "tokens": tokens,
            "pool": pool, "empty": empty, "ctx": ctx, "packed": packed, "shape": shape}


def _pages(name, kind, n, lo, hi, hkv, d, ps, planes, shape, pool=0, shared=0.0, spare=0.25):
    return {"name": name, "op": "pages", "kind": kind, "dtype": "bf16", "n": n, "lo": lo,
            "hi": hi, "hkv": hkv, "d": d, "ps": ps, "planes": planes, "pool": pool,
            "shared": shared, "spare": spare, "shape": shape}


def listed():
    return [
        # one user's chat, one token after a thousand: latency alone
        _attn("decode_single_1000", "decode", "bf16", 1, 1000, 1000, 32, 8, 128, 16, 1),
        # the ordinary decode batch: 64 users whose histories differ by two orders of size
        _attn("decode_batch_64", "decode", "bf16", 64, 64, 8192, 32, 16, 128, 64, 2,
              packed=True),
        # a few very long documents, wide heads, few key heads: one unit of work per key
        # head would leave most of the GPU idle
        _attn("decode_long_4", "decode", "f16", 4, 60001, 131071, 16, 2, 256, 32, 3),
        # half-full serving pool, sliding window with sinks, 32-bit cache, odd head ratio,
        # padding sequences that hold nothing
        _attn("decode_window_pool", "decode", "f32", 256, 1, 16384, 12, 4, 64, 16, 4,
              window=1024, sinks=4, pool=512, empty=3),
        # verification of four draft tokens of 64 users
        _attn("verify_64x4", "decode", "bf16", 64, 300, 8192, 16, 4, 128, 32, 5, tokens=4),
        # a ragged batch of fresh prompts, 16384 positions in all
        _attn("prompt_ragged_16k", "prompt", "bf16", 16384, 1, 4096, 32, 8, 128, 64, 6,
              packed=True),
        # four prompts of 4096 in a layer with a sliding window and sinks
        _attn("prompt_window_4x4096", "prompt", "f16", 4 * 4096, 4096, 4096, 16, 8, 64, 16, 7,
              window=1000, sinks=4),
        # one chunk of a long prompt: 1500 new positions after 30000 that are in the cache
        _attn("prompt_chunk_30k", "prompt", "bf16", 1500, 1500, 1500, 24, 2, 256, 128, 8,
              ctx=30000),
        # the decode step's new keys and values, and the ragged prompt's
        _attn("append_batch_64", "append", "bf16", 64, 64, 8192, 32, 16, 128, 64, 9,
              packed=True),
        _attn("append_ragged_16k", "append", "f16", 16384, 1, 4096, 32, 8, 128, 16, 10),
        # 64 users' chats each continued a second time from where they are
        _pages("pages_fork_64", "fork", 64, 100, 4096, 8, 128, 64, 8, 11, pool=128),
        # a pool with holes made dense
        _pages("pages_compact", "compact", 48, 300, 4096, 8, 128, 16, 8, 12, pool=128,
               shared=0.2, spare=0.5),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the same ranges: sizes log-uniform, odd ones among them."""
    op = rng.choice(["decode", "decode", "decode", "prompt", "prompt", "append", "pages"])
    ps = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    shape = rng.randrange(1 << 30)
    if op == "pages":
        kind = rng.choice(["copy", "reserve", "fork", "truncate", "compact"])
        n = _logint(rng, 1, 96)
        return _pages("", kind, n, 1, _logint(rng, 16, 8192), min(hkv, 8), min(d, 128), ps,
                      rng.choice([2, 4, 8]), shape, pool=2 * n,
                      shared=rng.choice([0.0, 0.3]), spare=rng.uniform(0.25, 0.6))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_logint(rng, 16, 4096), rng.choice([0, 1, 4]))])
    packed = rng.random() < 0.5
    if op == "append":
        n = _logint(rng, 1, 16384)
        return _attn("", op, dtype, n, 1, 4096, hkv * g, hkv, d, ps, shape, packed=packed)
    if op == "decode":
        n = _logint(rng, 1, 256)
        # a cache of at most 256 MB a plane bounds the longest history
        cap = max(64, (1 << 28) // (n * hkv * d * BYTES[dtype]))
        hi = min(131071, _logint(rng, 64, cap))
        tokens = rng.choice([1, 1, 1, 2, 4, 5])
        return _attn("", op, dtype, n, rng.choice([1, max(1, hi // 7)]), hi, hkv * g, hkv, d,
                     ps, shape, window=window, sinks=sinks, tokens=tokens,
                     pool=rng.choice([0, 2 * n]), empty=rng.choice([0, 1]) if n > 1 else 0,
                     packed=packed)
    # a prompt's cost grows with its length squared: the total is cut by heads and size
    if dtype == "f32":
        hkv = min(hkv, 4)
    total = _logint(rng, 16, max(64, 16384 * 32 * 128 // max(hkv * g * d, 32 * 128)))
    if dtype == "f32":
        total = max(1, total // 4)
    ctx = rng.choice([0, 0, _logint(rng, 1, 8192)])
    hi = min(4096, total)
    return _attn("", op, dtype, total, rng.choice([1, max(1, hi // 5)]), hi, hkv * g, hkv, d, ps,
                 shape, window=window, sinks=sinks, ctx=ctx, packed=packed)


# ------------------------------------------------------------------ sizes of a case

def _new_tokens(case):
    """New positions of every sequence."""
    if case["op"] == "decode":
        return [case["tokens"]] * case["n"]
    if case["op"] == "append" and case["n"] <= 256:
        return [1] * case["n"]
    rng, left, out = random.Random(case["shape"]), case["n"], []
    while left > 0:
        out.append(min(left, _logint(rng, case["lo"], case["hi"])))
        left -= out[-1]
    return out


def _lengths(case):
    """Length of every sequence once the new positions are in the cache."""
    rng = random.Random(case["shape"] + 1)
    new = _new_tokens(case)
    if case["op"] == "prompt":
        # chunks of prompts follow histories of up to ctx positions
        return [m + (case["ctx"] if len(new) == 1 or not case["ctx"]
                     else rng.randrange(case["ctx"] + 1)) for m in new]
    if case["op"] == "append" and case["n"] > 256:
        return [m + rng.randrange(100) for m in new]
    lens = [max(m, _logint(rng, case["lo"], case["hi"])) for m in new]
    for i in range(case["empty"]):
        lens[rng.randrange(len(lens))] = 0
    return lens


def _visible(case, p):
    """How many keys position p sees."""
    if p < 0:
        return 0
    if case["window"] <= 0 or case["window"] + case["sinks"] > p:
        return p + 1
    return case["window"] + case["sinks"]


def _pages_of(length, ps):
    return -(-length // ps)


def work(case):
    if case["op"] == "pages":
        return _pages_work(case)
    e, d, hq, hkv = BYTES[case["dtype"]], case["d"], case["hq"], case["hkv"]
    new, lens = _new_tokens(case), _lengths(case)
    rows = sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * 2 * rows * hkv * d * e + 4 * rows, "flops": 0}
    pairs = keys = table = 0
    for m, n in zip(new, lens):
        for p in range(n - m, n):
            pairs += _visible(case, p)
        first = max(0, n - m)
        lo = max(0, first - case["window"] + 1) if case["window"] > 0 else 0
        seen = n - lo + min(case["sinks"], lo)
        keys += seen
        table += _pages_of(seen, case["ps"])
    return {"bytes": 2 * keys * hkv * d * e + 2 * rows * hq * d * e + 4 * table + 4 * len(lens),
            "flops": 4 * pairs * hq * d}


def _pages_sizes(case):
    """(lengths of the live slots, live pages, pages in the pool) of a bookkeeping case."""
    rng = random.Random(case["shape"])
    lens = [_logint(rng, case["lo"], case["hi"]) for _ in range(case["n"])]
    live = sum(_pages_of(n, case["ps"]) for n in lens)
    n_pages = int(live / (1.0 - case["spare"])) + 2 * case["n"] + 1
    return lens, live, n_pages


def _pages_work(case):
    lens, live, n_pages = _pages_sizes(case)
    page = case["hkv"] * case["ps"] * case["d"] * BYTES[case["dtype"]] * case["planes"]
    kind, n = case["kind"], case["n"]
    if kind == "copy":
        return {"bytes": 2 * page * n + 8 * n, "flops": 0}
    if kind == "compact":
        moved = int(live * (n_pages - live) / n_pages)
        return {"bytes": 2 * page * moved + 8 * n_pages + 8 * live, "flops": 0}
    if kind == "fork":
        part = sum(1 for m in lens if m % case["ps"])
        return {"bytes": 2 * page * part + 16 * live + 8 * n, "flops": 0}
    if kind == "reserve":
        return {"bytes": 16 * n, "flops": 0}
    return {"bytes": 16 * live // 2 + 8 * n, "flops": 0}


# ------------------------------------------------------------------ inputs

def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _rows(gen, total, hq, hkv, d, dtype, packed):
    """q, k, v of every new position: apart, or slices of one projection's output."""
    if packed:
        qkv = _randn(gen, (total, hq + 2 * hkv, d), dtype)
        qkv[:, :hq] *= 2
        return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    return (2 * _randn(gen, (total, hq, d), dtype), _randn(gen, (total, hkv, d), dtype),
            _randn(gen, (total, hkv, d), dtype))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = random.Random(seed)
    return _prepare_pages(case, gen, host) if case["op"] == "pages" else \
        _prepare_attention(case, gen, host)


def _prepare_attention(case, gen, host):
    dtype, ps, hq, hkv, d = DTYPES[case["dtype"]], case["ps"], case["hq"], case["hkv"], case["d"]
    new, lens = _new_tokens(case), _lengths(case)
    n = len(lens)
    pool = case["pool"] or n
    slots = host.sample(range(pool), n) if case["pool"] else list(range(n))
    need = [_pages_of(m, ps) for m in lens]
    n_pages = sum(need) + sum(need) // 8 + 1
    max_pages = max(1, max(need))
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    rows = torch.full((pool, max_pages), -1, dtype=torch.int32, device="cuda")
    lens_pool = [0] * pool
    at = 0
    for s, m, length in zip(slots, need, lens):
        rows[s, :m] = ids[at:at + m]
        lens_pool[s] = length
        at += m
    q, k, v = _rows(gen, sum(new), hq, hkv, d, dtype, case["packed"])
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    st = {
        "case": case, "new": new, "lens": lens, "slots_host": slots, "cu_host": cu,
        "n_pages": n_pages, "max_pages": max_pages, "q": q, "k": k, "v": v,
        "k_pages": _randn(gen, (n_pages, hkv, ps, d), dtype),
        "v_pages": _randn(gen, (n_pages, hkv, ps, d), dtype),
        "table": rows, "kv_lens": torch.tensor(lens_pool, dtype=torch.int32, device="cuda"),
        "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
        "slots": torch.tensor(slots, dtype=torch.int32, device="cuda") if case["pool"] else None,
        "pool": pool, "out": torch.empty(sum(new), hq, d, dtype=dtype, device="cuda"),
        "scale": 1.0 / math.sqrt(d),
    }
    if own and case["op"] in ("decode", "prompt"):
        import gated_deltanet_linear_scan_gb300 as gdn
        size = (gdn.gdn_attn_decode_workspace_size(n, case["tokens"], hq, hkv, d)
                if case["op"] == "decode" else
                gdn.gdn_attn_prefill_workspace_size(n, sum(new), hq, hkv, d))
        st["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    return st


def _prepare_pages(case, gen, host):
    ps, n, pool = case["ps"], case["n"], case["pool"]
    lens, _, n_pages = _pages_sizes(case)
    max_pages = max(_pages_of(m, ps) for m in lens) + 1
    slots = host.sample(range(pool), n)
    rest = [s for s in range(pool) if s not in set(slots)]
    ids = iter(torch.randperm(n_pages, generator=gen, device="cuda").tolist())
    table = [[-1] * max_pages for _ in range(pool)]
    kv_lens, refs = [0] * pool, [0] * n_pages
    for i, (s, m) in enumerate(zip(slots, lens)):
        share = 0
        if i and host.random() < case["shared"]:
            # this sequence began as a fork of the one before it: full pages are shared
            share = min(m, lens[i - 1]) // ps
        for c in range(_pages_of(m, ps)):
            page = table[slots[i - 1]][c] if c < share else next(ids)
            table[s][c] = page
            refs[page] += 1
        kv_lens[s] = m
    elems = case["hkv"] * ps * case["d"]
    ints = dict(dtype=torch.int32, device="cuda")
    flat = [x for row in table for x in row] + kv_lens + refs
    st = {"case": case, "book": torch.tensor(flat, **ints), "n_pages": n_pages,
          "max_pages": max_pages, "page_bytes": elems * BYTES[case["dtype"]],
          "pages": _randn(gen, (case["planes"], n_pages, elems), DTYPES[case["dtype"]]),
          "slots": torch.tensor(slots, **ints), "children": torch.tensor(rest[:n], **ints)}
    if case["kind"] == "copy":
        free = [p for p in range(n_pages) if refs[p] == 0]
        used = [p for p in range(n_pages) if refs[p] > 0]
        m = min(n, len(free), len(used))
        st["src"] = torch.tensor(host.sample(used, m), **ints)
        st["dst"] = torch.tensor(host.sample(free, m), **ints)
    if case["kind"] == "reserve":
        st["count"] = torch.tensor([host.choice([0, 1, 1, 1, 4]) for _ in lens], **ints)
    if case["kind"] == "truncate":
        st["count"] = torch.tensor([host.choice([0, m // 2, max(0, m - 3)]) for m in lens],
                                   **ints)
    if own:
        import gated_deltanet_linear_scan_gb300 as gdn
        size = gdn.gdn_pages_workspace_size(pool, n_pages)
        st["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "pages":
        return _run_pages_own(state) if own else _run_pages(state)
    if case["op"] == "append":
        return _append_own(state) if own else _append(state)
    return _attention_own(state) if own else _attention(state)


def _append_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    gdn.gdn_kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"],
                      st["kv_lens"], st["cu"], len(st["lens"]), st["k"].shape[0], c["hkv"],
                      c["d"], c["ps"], st["n_pages"], st["max_pages"], slots=st["slots"],
                      pool=st["pool"])
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _attention_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    sizes = (c["hq"], c["hkv"], c["d"], c["ps"], st["n_pages"], st["max_pages"], c["window"],
             c["sinks"], st["scale"], st["ws"])
    if c["op"] == "decode":
        gdn.gdn_attn_decode(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                            st["out"], c["n"], c["tokens"], *sizes, slots=st["slots"],
                            pool=st["pool"])
    else:
        gdn.gdn_attn_prefill(st["q"], st["k_pages"], st["v_pages"], st["table"],
                             st["kv_lens"], st["out"], st["cu"], len(st["new"]),
                             st["q"].shape[0], max(st["new"]), *sizes, slots=st["slots"],
                             pool=st["pool"])
    return st["out"]


def _run_pages_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    table, kv_lens, refs = _book(st)
    data = (c["ps"], c["planes"], st["n_pages"], st["page_bytes"], st["max_pages"])
    kind = c["kind"]
    if kind == "copy":
        gdn.gdn_pages_copy(st["pages"], st["src"], st["dst"], st["src"].numel(), c["planes"],
                           st["n_pages"], st["page_bytes"])
    elif kind == "reserve":
        gdn.gdn_pages_reserve(st["pages"], table, kv_lens, refs, st["count"], c["n"], *data,
                              st["ws"], slots=st["slots"], pool=c["pool"])
    elif kind == "fork":
        gdn.gdn_pages_fork(st["pages"], table, kv_lens, refs, st["slots"], st["children"],
                           c["n"], *data, c["pool"], st["ws"])
    elif kind == "truncate":
        gdn.gdn_pages_truncate(table, kv_lens, refs, st["count"], c["n"], c["ps"],
                               st["n_pages"], st["max_pages"], slots=st["slots"],
                               pool=c["pool"])
        return {"table": table, "kv_lens": kv_lens, "refs": refs}
    else:
        gdn.gdn_pages_compact(st["pages"], table, kv_lens, refs, *data, c["pool"], st["ws"])
    return {"table": table, "kv_lens": kv_lens, "refs": refs, "pages": st["pages"]}


# ------------------------------------------------------------------ the plain forms

def _positions(st, n, pos):
    """Pages and rows inside them of the given positions of sequence n."""
    ps = st["case"]["ps"]
    page = st["table"][st["slots_host"][n]].long()[torch.div(pos, ps, rounding_mode="floor")]
    return page, pos % ps


def _append(st):
    for n, (m, length) in enumerate(zip(st["new"], st["lens"])):
        page, row = _positions(st, n, torch.arange(length - m, length, device="cuda"))
        a = st["cu_host"][n]
        st["k_pages"][page, :, row] = st["k"][a:a + m]
        st["v_pages"][page, :, row] = st["v"][a:a + m]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _attention(st):
    c = st["case"]
    hkv, d = c["hkv"], c["d"]
    g = c["hq"] // hkv
    for n, (m, length) in enumerate(zip(st["new"], st["lens"])):
        a = st["cu_host"][n]
        if length <= 0:
            st["out"][a:a + m] = 0
            continue
        # keys that some new position sees
        lo = max(0, length - m - c["window"] + 1) if c["window"] > 0 else 0
        pos = torch.arange(lo, length, device="cuda")
        if c["window"] > 0 and c["sinks"] > 0 and lo > 0:
            pos = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), pos])
        page, row = _positions(st, n, pos)
        k = st["k_pages"][page, :, row].float().permute(1, 2, 0)           # [hkv][d][keys]
        v = st["v_pages"][page, :, row].float().permute(1, 0, 2)           # [hkv][keys][d]
        step = max(1, (1 << 28) // (c["hq"] * pos.numel()))
        for b in range(0, m, step):
            e = min(m, b + step)
            q = st["q"][a + b:a + e].float().reshape(e - b, hkv, g, d)
            q = q.permute(1, 0, 2, 3).reshape(hkv, (e - b) * g, d)
            p = torch.arange(length - m + b, length - m + e, device="cuda")[:, None]
            see = pos <= p
            if c["window"] > 0:
                see = see & ((pos > p - c["window"]) | (pos < c["sinks"]))
            see = see.repeat_interleave(g, 0)
            s = torch.where(see, torch.matmul(q, k) * st["scale"], -math.inf)
            top = s.amax(-1, keepdim=True)
            w = torch.where(see, torch.exp(s - top), 0.0)
            total = w.sum(-1, keepdim=True)
            o = torch.where(total > 0, torch.matmul(w, v) / total, 0.0)
            o = o.reshape(hkv, e - b, g, d).permute(1, 0, 2, 3).reshape(e - b, hkv * g, d)
            st["out"][a + b:a + e] = o.to(st["out"].dtype)
    return st["out"]


def _book(st):
    """The bookkeeping of this pass: a copy, so that every pass starts from the same state."""
    c, book = st["case"], st["book"].clone()
    a = c["pool"] * st["max_pages"]
    return book[:a].view(c["pool"], st["max_pages"]), book[a:a + c["pool"]], book[a + c["pool"]:]


def _copy_pages(st, src, dst):
    st["pages"][:, dst] = st["pages"][:, src]


def _run_pages(st):
    c = st["case"]
    ps, kind = c["ps"], c["kind"]
    table, kv_lens, refs = _book(st)
    cols = torch.arange(st["max_pages"], device="cuda")[None, :]
    if kind == "copy":
        _copy_pages(st, st["src"].long(), st["dst"].long())
    elif kind == "fork":
        parents, children = st["slots"].long(), st["children"].long()
        lens = kv_lens[parents]
        full, part = (lens // ps)[:, None], (lens % ps > 0)
        free = torch.nonzero(refs == 0)[:, 0]
        mine = free[part.cumsum(0) - part.long()]
        rows = table[parents]
        last = rows.gather(1, full.long())[:, 0].long()
        shared = cols < full
        table[children] = torch.where(
            shared, rows, torch.where((cols == full) & part[:, None], mine[:, None], -1).int())
        kv_lens[children] = lens
        held = rows[shared].long()
        refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
        refs[mine[part]] = 1
        _copy_pages(st, last[part], mine[part])
    elif kind == "reserve":
        slots, count = st["slots"].long(), st["count"]
        lens = kv_lens[slots]
        old, end = (lens + ps - 1) // ps, (lens + count + ps - 1) // ps
        rows = table[slots]
        lastcol = (lens // ps).clamp(max=st["max_pages"] - 1).long()[:, None]
        last = rows.gather(1, lastcol)[:, 0]
        # a shared page that is only partly full is replaced by a copy before it is written
        cow = (lens % ps > 0) & (count > 0) & (refs[last.clamp(min=0).long()] > 1)
        need = end - old + cow.int()
        base = need.cumsum(0) - need
        free = torch.nonzero(refs == 0)[:, 0]
        fresh = (cols >= old[:, None]) & (cols < end[:, None])
        index = base[:, None] + cow.int()[:, None] + cols - old[:, None]
        take = torch.where(fresh, free[index.clamp(0, free.numel() - 1)].int(), rows)
        copy = free[base.clamp(0, free.numel() - 1)]
        take = torch.where((cols == lastcol) & cow[:, None], copy[:, None].int(), take)
        table[slots] = take
        kv_lens[slots] = lens + count
        refs[take[fresh].long()] = 1
        src, dst = last[cow].long(), copy[cow]
        refs.index_add_(0, src, -torch.ones_like(src, dtype=torch.int32))
        refs[dst] = 1
        _copy_pages(st, src, dst)
    elif kind == "truncate":
        slots, keep = st["slots"].long(), st["count"]
        lens = kv_lens[slots]
        rows = table[slots]
        gone = (cols >= ((keep + ps - 1) // ps)[:, None]) & (cols < ((lens + ps - 1) // ps)[:, None])
        held = rows[gone].long()
        refs.index_add_(0, held, -torch.ones_like(held, dtype=torch.int32))
        table[slots] = torch.where(gone, -1, rows)
        kv_lens[slots] = keep
        return {"table": table, "kv_lens": kv_lens, "refs": refs}
    else:
        live = refs > 0
        index = torch.arange(st["n_pages"], device="cuda")
        inside = index < live.sum()
        src = torch.nonzero(live & ~inside)[:, 0]
        dst = torch.nonzero(~live & inside)[:, 0]
        to = index.int()
        to[src] = dst.int()
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
        refs[dst] = refs[src]
        refs[src] = 0
        _copy_pages(st, src, dst)
    return {"table": table, "kv_lens": kv_lens, "refs": refs, "pages": st["pages"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] in ("append", "pages"):
        return None  # copies and whole numbers
    if work(case)["flops"] > 4e12:
        return None  # 64-bit arithmetic would take too long
    st = prepare(case, seed)
    hq, d, ps, window, sinks = case["hq"], case["d"], case["ps"], case["window"], case["sinks"]
    group = hq // case["hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for i, (m, length) in enumerate(zip(st["new"], st["lens"])):
        held = st["table"][st["slots_host"][i], :_pages_of(length, ps)].long()
        # [kv head][position][d], whole pages laid end to end and cut at the length
        keys, vals = (st[x][held].transpose(0, 1).reshape(case["hkv"], -1, d)[:, :length]
                      for x in ("k_pages", "v_pages"))
        at = 0
        while at < m and length > 0:
            end = min(m, at + max(1, (1 << 26) // length))
            p = torch.arange(length - m + at, length - m + end, device="cuda").view(-1, 1)
            j = torch.arange(length, device="cuda").view(1, -1)
            hidden = j > p
            if window > 0:
                hidden |= (j <= p - window) & (j >= sinks)
            dead = hidden.all(-1)
            for h in range(hq):
                q = st["q"][row + at:row + end, h].double()
                s = torch.einsum("td,kd->tk", q, keys[h // group].double()) / math.sqrt(d)
                s = s.masked_fill(hidden, -math.inf)
                logsum = torch.logsumexp(s, -1, keepdim=True)
                w = torch.exp(s - logsum).masked_fill(hidden, 0.0)
                o = torch.einsum("tk,kd->td", w, vals[h // group].double())
                out[row + at:row + end, h] = o.masked_fill(dead.view(-1, 1), 0.0)
            at = end
        row += m
    return out
