"""Workloads of the operators of a speculative step with a tree of drafts: their inputs, their
plain forms, their work.

A serving step may draft a tree of tokens for every sequence (up to 64 nodes, node 0 the token
that is certain) and have the model check all of them at once. Five operators:

  attn    attention of the tree's nodes over a sequence's paged cache: a node sees the cache
          and its own ancestors
  block   the Gated-DeltaNet block over the nodes: each continues its parent's state
  commit  the recurrent state and the conv history carried on along the accepted path
  accept  the accepted path, from the tokens sampled at the nodes, and the cache rows of its
          nodes moved together in every layer's planes
  sample  a token for every row of logits from one given uniform number: temperature, top-k,
          top-p, min-p

parents[n][i] is the parent of node i of sequence n: below i, or -1 where the node continues
the sequence itself, or -2 where there is no node. `run` computes in elementary torch
operations in 32 bits (sampling, whose tokens hang on which side of a border a sum falls, in
64), or, with `own` set, through the framework's entry points; `exact` is the definition in 64
bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
TURNS = 4  # sets of what a pass changes in place, taken in turn


# ------------------------------------------------------------------ the cases

def _attn(name, dtype, n, nodes, lo, hi, hq, hkv, d, ps, shape, window=0, sinks=0, pool=0,
          packed=False, ragged=False, chain=0.4):
    return {"name": name, "op": "attn", "dtype": dtype, "n": n, "nodes": nodes, "lo": lo,
            "hi": hi, "hq": hq, "hkv": hkv, "d": d, "ps": ps, "window": window, "sinks": sinks,
            "pool": pool, "packed": packed, "ragged": ragged, "chain": chain, "shape": shape}


def _block(name, op, n, nodes, hk, h, s, kernel, shape, pool=0, ragged=False, chain=0.4):
    return {"name": name, "op": op, "n": n, "nodes": nodes, "hk": hk, "h": h, "s": s,
            "kernel": kernel, "pool": pool, "ragged": ragged, "chain": chain, "shape": shape}


def _accept(name, n, nodes, lo, hi, hkv, d, ps, planes, shape, pool=0, ragged=False, chain=0.4):
    return {"name": name, "op": "accept", "dtype": "bf16", "n": n, "nodes": nodes, "lo": lo,
            "hi": hi, "hkv": hkv, "d": d, "ps": ps, "planes": planes, "pool": pool,
            "ragged": ragged, "chain": chain, "shape": shape}


def _sample(name, dtype, rows, vocab, kind, shape, per_set=1, pad=0, banned=0.0):
    return {"name": name, "op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab,
            "kind": kind, "per_set": per_set, "pad": pad, "banned": banned, "shape": shape}


def listed():
    return [
        # 64 users' trees of 16 drafts over histories that differ by two orders of size
        _attn("attn_batch_64x16", "bf16", 64, 16, 64, 8192, 32, 16, 128, 64, 1, packed=True),
        # eight long documents with the widest trees and many query heads a key head
        _attn("attn_long_8x64", "f16", 8, 64, 16001, 40000, 24, 4, 128, 32, 2, pool=16),
        # one user, a tree of 24 over 4000: latency
        _attn("attn_single_24", "bf16", 1, 24, 4000, 4000, 16, 4, 256, 16, 3),
        # a pool with a 32-bit cache, sliding window and sinks, odd head ratio, padded trees
        _attn("attn_window_pool", "f32", 96, 9, 9, 16384, 12, 4, 64, 16, 4, window=1024, sinks=4,
              pool=192, ragged=True),
        # the recurrent block over the 64 users' trees, at the benchmark's heads
        _block("block_64x16", "block", 64, 16, 16, 32, 128, 4, 5),
        # one user's tree of 48
        _block("block_single_48", "block", 1, 48, 16, 32, 128, 4, 6),
        # the states of the 64 users along their accepted paths; of one user
        _block("commit_64x16", "commit", 64, 16, 16, 32, 128, 4, 7),
        _block("commit_pool_5x63", "commit", 5, 63, 2, 6, 64, 3, 8, pool=11, ragged=True),
        # acceptance for the 64 users, 8 layers' planes; for one with a long tree
        _accept("accept_64x16", 64, 16, 64, 2048, 8, 128, 64, 16, 9, pool=128),
        _accept("accept_single_64", 1, 64, 3000, 3000, 4, 64, 16, 4, 10, chain=0.9),
        # one row, the ordinary settings
        _sample("sample_single", "bf16", 1, 128000, "top_p", 11),
        # every node of 64 trees of 16: 1024 rows, each user with settings of their own, of an
        # odd vocabulary whose rows are slices of padded ones
        _sample("sample_verify_64x16", "f32", 1024, 100003, "mixed", 12, per_set=16, pad=61,
                banned=0.2),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the same ranges: sizes log-uniform, odd ones among them."""
    op = rng.choice(["attn", "attn", "attn", "block", "block", "commit", "accept", "sample",
                     "sample"])
    shape = rng.randrange(1 << 30)
    nodes = _logint(rng, 1, 64)
    chain = rng.choice([0.0, 0.4, 0.8, 1.0])
    ragged = rng.random() < 0.4
    if op == "sample":
        dtype = rng.choice(["bf16", "f16", "f32"])
        vocab = _logint(rng, 1000, 262144)
        rows = _logint(rng, 1, max(1, min(1024, (400 << 20) // (vocab * BYTES[dtype]))))
        return _sample("", dtype, rows, vocab,
                       rng.choice(["greedy", "free", "top_k", "top_p", "min_p", "mixed"]), shape,
                       per_set=rng.choice([1, 1, 4]), pad=rng.choice([0, 0, 8, 5]),
                       banned=rng.choice([0.0, 0.0, 0.3]))
    if op in ("block", "commit"):
        s = rng.choice([32, 64, 128, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8, 16])
        h = hk * rng.choice([1, 2, 2, 3, 4])
        # at most 2 GB of states would be kept if every node had one
        n = _logint(rng, 1, max(1, min(64, (1 << 31) // (nodes * h * s * s * 4))))
        return _block("", op, n, nodes, hk, h, s, rng.choice([4, 4, 4, 2, 3, 6]), shape,
                      pool=rng.choice([0, 2 * n]), ragged=ragged, chain=chain)
    ps = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "accept":
        n = _logint(rng, 1, 96)
        return _accept("", n, nodes, nodes, nodes + _logint(rng, 8, 2048), min(hkv, 8),
                       rng.choice([64, 128]), ps, rng.choice([2, 4, 8, 16]), shape,
                       pool=rng.choice([0, 2 * n]), ragged=ragged, chain=chain)
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_logint(rng, 16, 4096), rng.choice([0, 1, 4]))])
    n = _logint(rng, 1, 128)
    # a cache of at most 256 MB a plane, and the work of the largest listed case, bound the
    # longest history
    cap = (1 << 28) // (n * hkv * d * BYTES[dtype])
    cap = min(cap, (1 << 32) // (n * nodes * hkv * group * d // (4 if dtype == "f32" else 1) + 1))
    hi = min(65536, nodes + _logint(rng, 64, max(65, cap)))
    return _attn("", dtype, n, nodes, rng.choice([nodes, max(nodes, hi // 7)]), hi, hkv * group,
                 hkv, d, ps, shape, window=window, sinks=sinks, pool=rng.choice([0, 2 * n]),
                 packed=rng.random() < 0.5, ragged=ragged, chain=chain)


# ------------------------------------------------------------------ sizes of a case

def _trees(case):
    """parents of every sequence: -1 for the root, -2 where a padded tree has no node."""
    rng = random.Random(case["shape"])
    out = []
    for _ in range(case["n"]):
        m = rng.randint(1, case["nodes"]) if case["ragged"] else case["nodes"]
        out.append([-1] + [i - 1 if rng.random() < case["chain"] else rng.randrange(i)
                           for i in range(1, m)] + [-2] * (case["nodes"] - m))
    return out


def _depths(tree):
    depth = []
    for p in tree:
        depth.append(-1 if p < -1 else 0 if p < 0 else depth[p] + 1)
    return depth


def _lengths(case):
    """Length of every sequence, its tree's nodes among them."""
    rng = random.Random(case["shape"] + 1)
    return [max(case["nodes"], _logint(rng, case["lo"], case["hi"])) for _ in range(case["n"])]


def _path_to(tree, i):
    out = []
    while i >= 0:
        out.append(i)
        i = tree[i]
    return out[::-1]


def _leaves(case):
    """The last accepted node of every sequence."""
    rng = random.Random(case["shape"] + 2)
    return [rng.randrange(sum(p > -2 for p in tree)) for tree in _trees(case)]


def _pages_of(length, ps):
    return -(-length // ps)


def work(case):
    op = case["op"]
    if op == "sample":
        sets = -(-case["rows"] // case["per_set"])
        return {"bytes": case["rows"] * (case["vocab"] * BYTES[case["dtype"]] + 8) + 16 * sets,
                "flops": 4 * case["rows"] * case["vocab"]}
    trees = _trees(case)
    depths = [_depths(t) for t in trees]
    nodes = sum(sum(x >= 0 for x in d) for d in depths)
    pairs = sum(sum(x + 1 for x in d) for d in depths)  # (node, itself or an ancestor)
    if op == "attn":
        e, d, hq, hkv = BYTES[case["dtype"]], case["d"], case["hq"], case["hkv"]
        w, sinks = case["window"], case["sinks"]
        keys = seen = table = 0
        for tree, depth, length in zip(trees, depths, _lengths(case)):
            base = length - case["nodes"]
            for x in depth:
                if x >= 0:  # of the cache before the tree; its ancestors are in `pairs`
                    seen += base if not w else min(base, max(0, w - 1 - x) + min(sinks, base))
            near = base if not w else min(base, w - 1 + sinks)
            keys += near + sum(x >= 0 for x in depth)
            table += _pages_of(near + case["nodes"], case["ps"])
        return {"bytes": 2 * keys * hkv * d * e + 2 * nodes * hq * d * e + 4 * table,
                "flops": 4 * (seen + pairs) * hq * d}
    if op == "accept":
        row = case["hkv"] * case["d"] * BYTES[case["dtype"]] * case["planes"]
        moved = 0
        for tree, last in zip(trees, _leaves(case)):
            moved += sum(i != j for i, j in enumerate(_path_to(tree, last)))
        return {"bytes": 2 * moved * row + 12 * case["n"] * case["nodes"] + 16 * case["n"],
                "flops": 0}
    n, hk, h, s, k = case["n"], case["hk"], case["h"], case["s"], case["kernel"]
    width = (2 * hk + h) * s
    state, conv = n * h * s * s, n * width * (k - 1)
    if op == "commit":
        kept = sum(len(_path_to(t, i)) for t, i in zip(trees, _leaves(case)))
        return {"bytes": 4 * (2 * state + 2 * conv + kept * (hk + h) * s),
                "flops": 2 * kept * h * s * s}
    return {"bytes": 4 * (state + conv + nodes * (width + 2 * h * s + 2 * h) + width * k),
            "flops": 4 * nodes * h * s * s + pairs * (4 * hk * s + 4 * h * s)}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = random.Random(seed)
    op = case["op"]
    if op == "sample":
        return _prepare_sample(case, gen, host)
    trees = _trees(case)
    st = {"case": case, "trees": trees, "parents": _ints(trees)}
    if op in ("attn", "accept"):
        _prepare_cache(case, gen, host, st)
    else:
        _prepare_block(case, gen, host, st)
    if op in ("accept", "commit"):
        _prepare_path(case, gen, host, st)
    return st


def _slots(case, host):
    return host.sample(range(case["pool"]), case["n"]) if case["pool"] else list(range(case["n"]))


def _prepare_cache(case, gen, host, st):
    dtype, ps, hkv, d = DTYPES[case["dtype"]], case["ps"], case["hkv"], case["d"]
    n, nodes, lens = case["n"], case["nodes"], _lengths(case)
    pool, slots = case["pool"] or n, _slots(case, host)
    need = [_pages_of(m, ps) for m in lens]
    n_pages, max_pages = sum(need) + sum(need) // 8 + 1, max(need)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((pool, max_pages), -1, dtype=torch.int32, device="cuda")
    held, at = [0] * pool, 0
    for s, m, length in zip(slots, need, lens):
        table[s, :m] = ids[at:at + m]
        held[s] = length
        at += m
    st.update(lens=lens, slots_host=slots, n_pages=n_pages, max_pages=max_pages, table=table,
              kv_lens=_ints(held), slots=_ints(slots) if case["pool"] else None, pool=pool)
    if case["op"] == "accept":
        st["turns"] = [_randn(gen, case["planes"], n_pages, hkv, ps, d, dtype=dtype)]
        st["turns"] += [st["turns"][0].clone() for _ in range(TURNS - 1)]
        return
    hq = case["hq"]
    if case["packed"]:
        st["q"] = _randn(gen, n * nodes, hq + 2 * hkv, d, dtype=dtype)[:, :hq]
    else:
        st["q"] = _randn(gen, n * nodes, hq, d, dtype=dtype)
    st["q"] *= 2
    st["k_pages"] = _randn(gen, n_pages, hkv, ps, d, dtype=dtype)
    st["v_pages"] = _randn(gen, n_pages, hkv, ps, d, dtype=dtype)
    st["out"] = torch.empty(n * nodes, hq, d, dtype=dtype, device="cuda")
    st["scale"] = 1.0 / math.sqrt(d)
    if own:
        import gated_deltanet_linear_scan_gb300 as gdn
        size = gdn.gdn_attn_tree_workspace_size(n, nodes, hq, hkv, d)
        st["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")


def _prepare_block(case, gen, host, st):
    n, t, hk, h, s, k = (case[x] for x in ("n", "nodes", "hk", "h", "s", "kernel"))
    pool, width = case["pool"] or n, (2 * hk + h) * s
    slots = _slots(case, host)
    a = -torch.exp(torch.rand(h, generator=gen, device="cuda") - 0.5)
    dt = 0.5 * _randn(gen, h)
    # the gate's logits, such that the log-decay is uniform in (-2, -0.01)
    g = -0.01 - 1.99 * torch.rand(n, t, h, generator=gen, device="cuda")
    st.update(slots_host=slots, slots=_ints(slots) if case["pool"] else None, pool=pool,
              qkv=_randn(gen, n, t, width), conv_w=0.5 * _randn(gen, width, k), a=a, dt=dt,
              alpha=torch.log(torch.expm1(g / a)) - dt, b=_randn(gen, n, t, h),
              z=_randn(gen, n, t, h, s), norm_w=1 + 0.1 * _randn(gen, s),
              conv_state=_randn(gen, pool, width, k - 1), state=0.1 * _randn(gen, pool, h, s, s),
              out=torch.empty(n, t, h, s, device="cuda"), scale=1 / math.sqrt(s), eps=1e-6)
    if own:
        import gated_deltanet_linear_scan_gb300 as gdn
        sizes = (n, t, hk, h, s)
        for name, size in (("tape", gdn.gdn_block_tree_tape_size(*sizes)),
                           ("ws", gdn.gdn_block_tree_workspace_size(*sizes))):
            st[name] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")


def _prepare_path(case, gen, host, st):
    """What the step before has left: the tokens drafted and sampled, or the block's tape."""
    leaves = _leaves(case)
    st["leaves"] = leaves
    if case["op"] == "accept":
        tokens, sampled = [], []
        for tree, last in zip(st["trees"], leaves):
            # drafts of one parent differ; what was sampled agrees along the path, and not
            # behind its end
            drafts = [7 * i + host.randrange(7) for i in range(len(tree))]
            picked = [10000 + host.randrange(1000) for _ in tree]
            path = _path_to(tree, last)
            for i, j in zip(path, path[1:]):
                picked[i] = drafts[j]
            tokens.append(drafts)
            sampled.append(picked)
        n, t = case["n"], case["nodes"]
        st.update(tokens=_ints(tokens), sampled=_ints(sampled), path=_ints([[0] * t] * n),
                  counts=_ints([[0] * n] * 4))
        return
    st["accepted"] = _ints([i + 1 for i in leaves])
    st["turns"] = [(st["state"].clone(), st["conv_state"].clone()) for _ in range(TURNS)]
    if own:
        _block_own(st)
    else:
        _, st["k"], st["g"], st["u"] = _block_plain(st)


def _prepare_sample(case, gen, host):
    dtype, rows, vocab = DTYPES[case["dtype"]], case["rows"], case["vocab"]
    x = _randn(gen, rows, vocab + case["pad"])
    # rows of different sharpness: some hundred likely tokens stand out of the bulk
    x *= 1.0 + 1.5 * torch.rand(rows, 1, generator=gen, device="cuda")
    likely = torch.randint(vocab, (rows, 200), generator=gen, device="cuda")
    x.scatter_add_(1, likely, 12 * torch.rand(rows, 200, generator=gen, device="cuda"))
    if case["banned"]:
        x[torch.rand(x.shape, generator=gen, device="cuda") < case["banned"]] = -math.inf
    sets = -(-rows // case["per_set"])
    temperature, top_k, top_p, min_p = [], [], [], []
    for _ in range(sets):
        kind = case["kind"] if case["kind"] != "mixed" else host.choice(
            ["greedy", "free", "top_k", "top_p", "top_p", "min_p", "all"])
        temperature.append(0.0 if kind == "greedy" else host.choice([0.6, 0.8, 1.0, 1.3]))
        top_k.append(_logint(host, 1, 1000) if kind in ("top_k", "all") else 0)
        top_p.append(host.uniform(0.5, 0.99) if kind in ("top_p", "all") else 1.0)
        min_p.append(host.choice([0.02, 0.05, 0.1]) if kind in ("min_p", "all") else 0.0)
    floats = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    return {"case": case, "logits": x.to(dtype)[:, :vocab], "temperature": floats(temperature),
            "top_k": _ints(top_k), "top_p": floats(top_p), "min_p": floats(min_p),
            "u": torch.rand(rows, generator=gen, device="cuda"),
            "tokens": torch.empty(rows, dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _attn_own, "block": _block_own, "commit": _commit_own,
                "accept": _accept_own, "sample": _sample_own}[op](state)
    if op == "block":
        return _block_plain(state)[0]
    return {"attn": _attn_plain, "commit": _commit_plain, "accept": _accept_plain,
            "sample": _sample_plain}[op](state)


def _turn(st):
    """The next set of what a pass changes in place."""
    st["turn"] = (st.get("turn", -1) + 1) % TURNS
    return st["turns"][st["turn"]]


def _attn_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    gdn.gdn_attn_tree(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                      st["out"], st["parents"], c["n"], c["nodes"], c["hq"], c["hkv"], c["d"],
                      c["ps"], st["n_pages"], st["max_pages"], c["window"], c["sinks"],
                      st["scale"], st["ws"], slots=st["slots"], pool=st["pool"])
    return st["out"]


def _block_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    gdn.gdn_block_tree(st["qkv"], st["conv_w"], st["conv_state"], st["alpha"], st["b"], st["dt"],
                       st["a"], st["z"], st["norm_w"], st["state"], st["out"], st["parents"],
                       c["n"], c["nodes"], c["hk"], c["h"], c["s"], c["kernel"], st["scale"],
                       st["eps"], st["eps"], st["tape"], st["ws"], slots=st["slots"],
                       pool=st["pool"])
    return st["out"]


def _commit_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    state, conv_state = _turn(st)
    gdn.gdn_block_tree_commit(st["qkv"], conv_state, state, st["parents"], st["accepted"], c["n"],
                              c["nodes"], c["hk"], c["h"], c["s"], c["kernel"], st["tape"],
                              slots=st["slots"], pool=st["pool"])
    return {"state": state, "conv_state": conv_state}


def _accept_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c, pages = st["case"], _turn(st)
    accepted, n_kept, new_lens, next_tokens = st["counts"]
    gdn.gdn_tree_accept(st["parents"], st["tokens"], st["sampled"], accepted, n_kept, new_lens,
                        next_tokens, st["path"], c["n"], c["nodes"], pages, st["table"],
                        st["kv_lens"], c["hkv"], c["ps"], c["planes"], st["n_pages"],
                        pages.stride(1) * pages.element_size(), st["max_pages"],
                        slots=st["slots"], pool=st["pool"])
    return {"pages": pages, "path": st["path"], "counts": st["counts"]}


def _sample_own(st):
    import gated_deltanet_linear_scan_gb300 as gdn
    c = st["case"]
    gdn.gdn_sample(st["logits"], st["u"], st["tokens"], c["rows"], c["vocab"],
                   temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                   min_p=st["min_p"], rows_per_set=c["per_set"])
    return st["tokens"]


# ------------------------------------------------------------------ the plain forms

def _above(trees):
    """above[n][i][j]: node j is node i, or an ancestor of it; depth[n][i]: -1 without a node."""
    n, t = len(trees), len(trees[0])
    above = torch.zeros(n, t, t, dtype=torch.bool)
    for x, tree in enumerate(trees):
        for i, p in enumerate(tree):
            if p >= 0:
                above[x, i] = above[x, p]
            if p > -2:
                above[x, i, i] = True
    return above.cuda(), above.sum(-1).cuda() - 1


def _attn_plain(st):
    c = st["case"]
    t, hkv, d, ps = c["nodes"], c["hkv"], c["d"], c["ps"]
    g, w = c["hq"] // hkv, c["window"]
    above, depth = _above(st["trees"])
    for n, length in enumerate(st["lens"]):
        base = length - t
        lo = max(0, base - w + 1) if w > 0 else 0
        key = torch.arange(lo, length, device="cuda")
        if w > 0 and c["sinks"] > 0 and lo > 0:
            key = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), key])
        page = st["table"][st["slots_host"][n]].long()[torch.div(key, ps, rounding_mode="floor")]
        k = st["k_pages"][page, :, key % ps].float().permute(1, 2, 0)
        v = st["v_pages"][page, :, key % ps].float().permute(1, 0, 2)
        # positions of the keys: a node's is its parent's and one
        node = (key - base).clamp(min=0)
        at = torch.where(key < base, key, base + depth[n][node])
        p = (base + depth[n])[:, None]
        see = (key < base)[None, :] | above[n][:, node]
        if w > 0:
            see = see & ((p - at < w) | (at < c["sinks"]))
        see = see & (depth[n] >= 0)[:, None]
        see = see.repeat_interleave(g, 0)
        q = st["q"][n * t:(n + 1) * t].float().reshape(t, hkv, g, d)
        q = q.permute(1, 0, 2, 3).reshape(hkv, t * g, d)
        s = torch.where(see, torch.matmul(q, k) * st["scale"], -math.inf)
        top = s.amax(-1, keepdim=True)
        e = torch.where(see, torch.exp(s - top), 0.0)
        total = e.sum(-1, keepdim=True)
        o = torch.where(total > 0, torch.matmul(e, v) / total, 0.0)
        o = o.reshape(hkv, t, g, d).permute(1, 0, 2, 3).reshape(t, hkv * g, d)
        st["out"][n * t:(n + 1) * t] = o.to(st["out"].dtype)
    return st["out"]


def _histories(st):
    """Raw inputs with the conv history in front, [n][K-1+nodes][C], and for each of them the one
    before it on its path."""
    c = st["case"]
    k = c["kernel"]
    slots = torch.tensor(st["slots_host"], device="cuda")
    rows = torch.cat([st["conv_state"][slots].transpose(1, 2), st["qkv"]], 1)
    up = st["parents"].long()
    up = torch.where(up >= 0, up + k - 1, k - 2)
    first = (torch.arange(k - 1, device="cuda") - 1).clamp(min=0)
    return rows, torch.cat([first[None].expand(c["n"], -1), up], 1)


def _block_plain(st):
    """(out, k, g, u): the block over the nodes, one after the other, each from its parent's
    state; and what the states change by."""
    c = st["case"]
    n, t, hk, h, s, kernel = (c[x] for x in ("n", "nodes", "hk", "h", "s", "kernel"))
    rows, up = _histories(st)
    at = torch.arange(t, device="cuda")[None].expand(n, -1) + kernel - 1
    pre = 0.0
    for tap in range(kernel - 1, -1, -1):
        pre = pre + torch.take_along_dim(rows, at[..., None], 1) * st["conv_w"][:, tap]
        at = torch.take_along_dim(up, at, 1)
    x = pre / (1 + torch.exp(-pre))
    q, k, v = x.split((hk * s, hk * s, h * s), -1)
    q, k = (y.reshape(n, t, hk, s) for y in (q, k))
    q, k = (y / torch.sqrt((y * y).sum(-1, keepdim=True)).clamp(min=st["eps"]) for y in (q, k))
    qh, kh = (y.repeat(1, 1, h // hk, 1) for y in (q, k))  # v-head i reads k-head i % hk
    v = v.reshape(n, t, h, s)
    soft = st["alpha"] + st["dt"]
    soft = torch.where(soft > 20, soft, torch.log1p(torch.exp(soft.clamp(max=20))))
    g = st["a"] * soft
    beta = 1 / (1 + torch.exp(-st["b"]))
    u, y = torch.zeros_like(v), torch.zeros_like(v)
    step = max(1, (1 << 32) // ((t + 1) * h * s * s * 4))
    for a in range(0, n, step):
        part = slice(a, min(n, a + step))
        m = part.stop - a
        states = torch.zeros(m, t + 1, h, s, s, device="cuda")
        states[:, 0] = st["state"][torch.tensor(st["slots_host"][part], device="cuda")]
        each = torch.arange(m, device="cuda")
        for i in range(t):
            up_i = (st["parents"][part, i].long() + 1).clamp(min=0)
            now = states[each, up_i] * torch.exp(g[part, i])[..., None, None]
            ki = kh[part, i][:, :, None, :]
            u[part, i] = (v[part, i] - (now * ki).sum(-1)) * beta[part, i][..., None]
            now = now + u[part, i][..., None] * ki
            states[:, i + 1] = now
            y[part, i] = st["scale"] * (now * qh[part, i][:, :, None, :]).sum(-1)
    out = y / torch.sqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * st["norm_w"]
    out = out * (st["z"] / (1 + torch.exp(-st["z"])))
    there = st["parents"] > -2
    st["out"].copy_(torch.where(there[..., None, None], out, 0.0))
    return st["out"], k, g, u


def _commit_plain(st):
    c = st["case"]
    state, conv_state = _turn(st)
    r, taps = c["h"] // c["hk"], c["kernel"] - 1
    for n, (slot, tree, last) in enumerate(zip(st["slots_host"], st["trees"], st["leaves"])):
        path = torch.tensor(_path_to(tree, last), device="cuda")
        g, u = st["g"][n, path], st["u"][n, path]
        k = st["k"][n, path].repeat(1, r, 1)
        # from behind a node to the path's end
        rest = g.flip(0).cumsum(0).flip(0)
        after = torch.exp(rest - g)
        now = torch.matmul((u * after[..., None]).permute(1, 2, 0), k.permute(1, 0, 2))
        state[slot] = state[slot] * torch.exp(rest[0])[:, None, None] + now
        rows = torch.cat([conv_state[slot].T, st["qkv"][n, path]])
        conv_state[slot] = rows[rows.shape[0] - taps:].T
    return {"state": state, "conv_state": conv_state}


def _accept_plain(st):
    c, pages = st["case"], _turn(st)
    n, t, ps = c["n"], c["nodes"], c["ps"]
    slots = torch.tensor(st["slots_host"], device="cuda")
    at = torch.zeros(n, 1, dtype=torch.long, device="cuda")
    path = torch.full((n, t), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    kept = torch.ones(n, 1, dtype=torch.long, device="cuda")
    going = torch.ones(n, 1, dtype=torch.bool, device="cuda")
    nodes = torch.arange(t, device="cuda")
    for i in range(1, t):
        child = (st["parents"] == at) & (st["tokens"] == st["sampled"].gather(1, at))
        first = torch.where(child, nodes, t).amin(1, keepdim=True)
        going = going & (first < t)
        at = torch.where(going, first, at)
        path[:, i] = torch.where(going, first, -1)[:, 0]
        kept = kept + going
    st["path"].copy_(path)
    base = st["kv_lens"][slots].long() - t
    st["counts"].copy_(torch.stack([at[:, 0] + 1, kept[:, 0], base + kept[:, 0],
                                    st["sampled"].gather(1, at)[:, 0].long()]))
    seq, to = torch.nonzero(path >= 0, as_tuple=True)
    row = lambda x: (st["table"][slots[seq], torch.div(x, ps, rounding_mode="floor")].long(), x % ps)  # noqa: E731
    src, dst = row(base[seq] + path[seq, to]), row(base[seq] + to)
    pages[:, dst[0], :, dst[1]] = pages[:, src[0], :, src[1]]
    return {"pages": pages, "path": st["path"], "counts": st["counts"]}


def _sample_plain(st):
    c = st["case"]
    rows, step = c["rows"], max(1, (1 << 25) // c["vocab"])
    ranks = torch.arange(c["vocab"], device="cuda")
    for a in range(0, rows, step):
        b = min(rows, a + step)
        group = torch.arange(a, b, device="cuda") // c["per_set"]
        t, k, p, m = (st[x][group][:, None] for x in ("temperature", "top_k", "top_p", "min_p"))
        x = st["logits"][a:b].double()
        x = torch.where(x.isnan(), -math.inf, x)
        order = x.sort(dim=-1, descending=True, stable=True)
        top = order.values[:, :1]
        w = torch.where(order.values == top, 1.0,
                        torch.exp((order.values - top) / torch.where(t > 0, t, 1.0).double()))
        keep = (ranks < torch.where(k > 0, k, c["vocab"])) & (order.values > -math.inf)
        w = torch.where(keep, w, 0.0)
        before = w.cumsum(-1) - w  # weight of the ranks above
        nucleus = (before < p.double() * w.sum(-1, keepdim=True)) | (p >= 1)
        keep = keep & nucleus & (w >= m.double()) & (t > 0)
        w = torch.where(keep | (ranks == 0), w, 0.0)
        by_index = torch.zeros_like(w).scatter_(1, order.indices, w).cumsum(-1)
        target = st["u"][a:b, None].double() * by_index[:, -1:]
        token = (by_index <= target).sum(-1)
        token = torch.where(top[:, 0] > -math.inf, token, -1)
        st["tokens"][a:b] = token.int()
    return st["tokens"]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] in ("accept", "sample"):
        return None  # copies and whole numbers
    if work(case)["flops"] > 2e12:
        return None  # 64-bit arithmetic would take too long
    st = prepare(case, seed)
    return _exact_attn(case, st) if case["op"] == "attn" else _exact_block(case, st)


def _exact_attn(case, st):
    t, hq, d, ps, window = (case[x] for x in ("nodes", "hq", "d", "ps", "window"))
    group = hq // case["hkv"]
    out = torch.zeros(case["n"] * t, hq, d, dtype=torch.float64, device="cuda")
    for n, (tree, length) in enumerate(zip(st["trees"], st["lens"])):
        held = st["table"][st["slots_host"][n], :_pages_of(length, ps)].long()
        keys, vals = (st[x][held].transpose(0, 1).reshape(case["hkv"], -1, d)[:, :length]
                      for x in ("k_pages", "v_pages"))
        base, depth = length - t, _depths(tree)
        pos = torch.arange(length, device="cuda")
        pos[base:] = base + torch.tensor(depth, device="cuda")
        hidden = torch.ones(t, length, dtype=torch.bool)
        for i in range(t):
            if depth[i] >= 0:
                hidden[i, :base] = False
                hidden[i, [base + j for j in _path_to(tree, i)]] = False
        hidden = hidden.cuda()
        if window > 0:
            mine = pos[base:].view(-1, 1)
            hidden |= (pos <= mine - window) & (pos >= case["sinks"])
        dead = hidden.all(-1)
        for h in range(hq):
            q = st["q"][n * t:(n + 1) * t, h].double()
            s = torch.einsum("td,kd->tk", q, keys[h // group].double()) / math.sqrt(d)
            s = s.masked_fill(hidden, -math.inf)
            w = torch.exp(s - torch.logsumexp(s, -1, keepdim=True)).masked_fill(hidden, 0.0)
            o = torch.einsum("tk,kd->td", w, vals[h // group].double())
            out[n * t:(n + 1) * t, h] = o.masked_fill(dead.view(-1, 1), 0.0)
    return out


def _exact_block(case, st):
    """One sequence after the other, path by path: the block as single tokens would run it."""
    hk, h, s, taps = case["hk"], case["h"], case["s"], case["kernel"] - 1
    f = lambda name: st[name].double()  # noqa: E731
    w, a, dt, norm_w = f("conv_w"), f("a"), f("dt"), f("norm_w")
    head = torch.arange(h, device="cuda") % hk
    out = torch.zeros(case["n"], case["nodes"], h, s, dtype=torch.float64, device="cuda")
    state = f("state") if case["op"] == "commit" else None
    conv = f("conv_state") if case["op"] == "commit" else None

    def step(n, i, big, hist):
        """(state, history, output) behind node i, from those of its parent."""
        taps_in = torch.cat([hist, f_qkv[n, i][:, None]], 1)
        pre = (taps_in * w).sum(1)
        x = pre * torch.sigmoid(pre)
        unit = lambda y: y / y.norm(dim=-1, keepdim=True).clamp(min=st["eps"])  # noqa: E731
        q, k = unit(x[:hk * s].view(hk, s))[head], unit(x[hk * s:2 * hk * s].view(hk, s))[head]
        v = x[2 * hk * s:].view(h, s)
        decay = torch.exp(a * torch.nn.functional.softplus(f_alpha[n, i] + dt))
        big = big * decay[:, None, None]
        delta = (v - torch.einsum("hji,hi->hj", big, k)) * torch.sigmoid(f_b[n, i])[:, None]
        big = big + torch.einsum("hj,hi->hji", delta, k)
        y = st["scale"] * torch.einsum("hji,hi->hj", big, q)
        z = f_z[n, i]
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * norm_w * z * torch.sigmoid(z)
        return big, taps_in[:, 1:], y

    f_qkv, f_alpha, f_b, f_z = f("qkv"), f("alpha"), f("b"), f("z")
    for n, (slot, tree) in enumerate(zip(st["slots_host"], st["trees"])):
        start = (st["state"][slot].double(), st["conv_state"][slot].double())
        if case["op"] == "commit":
            big, hist = start
            for i in _path_to(tree, st["leaves"][n]):
                big, hist, _ = step(n, i, big, hist)
            state[slot], conv[slot] = big, hist
            continue
        after = {-1: start}
        last_use = {p: i for i, p in enumerate(tree)}
        for i, p in enumerate(tree):
            if p < -1:
                continue
            big, hist, out[n, i] = step(n, i, *after[p])
            after[i] = (big, hist)
            for x in [x for x in after if last_use.get(x, -1) <= i and x != i]:
                del after[x]
    return {"state": state, "conv_state": conv} if case["op"] == "commit" else out
