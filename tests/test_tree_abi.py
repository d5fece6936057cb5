"""Host-side refusals of the calls on trees of drafts (no GPU needed): every bad argument gives its
documented status before anything is enqueued, and calls with nothing to do are no-ops."""
import pytest

import gated_deltanet_linear_scan_gb300 as gdn

OK, NULL, SHAPE, UNSUP, ALIGN = 0, 1, 2, 3, 4
P, MIS = 0x10000, 0x10004  # fake device addresses, aligned and not; never dereferenced here
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    gdn.build_if_needed()
    return gdn.library()


def attn(lib, q=P, kp=P, vp=P, table=P, lens=P, out=P, parents=P, n=2, nodes=5, hq=4, hkv=2, d=64,
         ps=16, n_pages=8, max_pages=4, window=0, sinks=0, qs=None, dtype=2, slots=None, pool=2, ws=P,
         ws_bytes=BIG):
    return lib.gdn_attn_tree(q, kp, vp, table, lens, out, parents, n, nodes, hq, hkv, d, ps, n_pages,
                             max_pages, window, sinks, 0.1, hq * d if qs is None else qs, dtype, slots,
                             pool, None, ws, ws_bytes, None)


def block(lib, n=2, nodes=5, hk=2, h=4, s=64, kernel=4, slots=None, pool=2, tape=P, tape_bytes=BIG,
          ws=P, ws_bytes=BIG, parents=P, **ptrs):
    names = ("qkv", "conv_w", "conv_state", "alpha", "b", "dt", "a", "z", "norm_w", "state", "out")
    assert set(ptrs) <= set(names)
    return lib.gdn_block_tree(*[ptrs.get(x, P) for x in names], parents, n, nodes, hk, h, s, kernel, 0.1,
                              1e-6, 1e-6, slots, pool, None, tape, tape_bytes, ws, ws_bytes, None)


def commit(lib, qkv=P, conv_state=P, state=P, parents=P, accepted=P, n=2, nodes=5, hk=2, h=4, s=64,
           kernel=4, slots=None, pool=2, tape=P, tape_bytes=BIG):
    return lib.gdn_block_tree_commit(qkv, conv_state, state, parents, accepted, n, nodes, hk, h, s,
                                     kernel, slots, pool, None, tape, tape_bytes, None)


def accept(lib, parents=P, tokens=P, sampled=P, accepted=P, n_kept=P, new_lens=P, next_tokens=P,
           path=P, n=2, nodes=5, pages=P, table=P, lens=P, hkv=2, ps=16, planes=2, n_pages=8, pb=4096,
           max_pages=4, slots=None, pool=2):
    return lib.gdn_tree_accept(parents, tokens, sampled, accepted, n_kept, new_lens, next_tokens, path,
                               n, nodes, pages, table, lens, hkv, ps, planes, n_pages, pb, max_pages,
                               slots, pool, None, None)


def sample(lib, logits=P, u=P, temperature=P, top_k=P, top_p=P, min_p=P, tokens=P, rows=3, vocab=100,
           stride=None, dtype=0, per_set=1):
    return lib.gdn_sample(logits, u, temperature, top_k, top_p, min_p, tokens, rows, vocab,
                          vocab if stride is None else stride, dtype, per_set, None, None)


@pytest.mark.parametrize("call", [attn, block, commit, accept])
def test_tree_arguments(lib, call):
    assert call(lib, parents=None) == NULL
    assert call(lib, n=-1) == SHAPE
    assert call(lib, nodes=0) == SHAPE
    assert call(lib, nodes=65) == UNSUP
    assert call(lib, pool=1) == SHAPE                # no slots and pool < n_seqs
    assert call(lib, slots=P, pool=0) == SHAPE
    assert call(lib, n=0) == OK


def test_attn_arguments(lib):
    for name in ("q", "kp", "vp", "table", "lens", "out", "ws"):
        assert attn(lib, **{name: None}) == NULL
    assert attn(lib, hq=5) == SHAPE
    assert attn(lib, hq=0) == SHAPE
    assert attn(lib, hkv=0) == SHAPE
    assert attn(lib, window=-1) == SHAPE
    assert attn(lib, sinks=-1) == SHAPE
    assert attn(lib, n_pages=0) == SHAPE
    assert attn(lib, max_pages=0) == SHAPE
    assert attn(lib, ps=24) == UNSUP
    assert attn(lib, d=96) == UNSUP
    assert attn(lib, dtype=3) == UNSUP
    assert attn(lib, n_pages=1 << 30) == UNSUP
    assert attn(lib, max_pages=1 << 30) == UNSUP
    assert attn(lib, qs=255) == SHAPE
    assert attn(lib, qs=260) == ALIGN
    for name in ("q", "kp", "vp", "out", "ws"):
        assert attn(lib, **{name: MIS}) == ALIGN
    size = lib.gdn_attn_tree_workspace_size
    for hq, hkv, d, dtype in ((4, 2, 64, 2), (40, 2, 256, 1), (12, 12, 128, 0)):
        need = size(2, 5, hq, hkv, d)
        assert need > 0 and attn(lib, hq=hq, hkv=hkv, d=d, dtype=dtype, ws_bytes=need - 1) == SHAPE
    assert size(2, 5, 5, 2, 64) == size(2, 5, 4, 2, 48) == size(2, 0, 4, 2, 64) == size(2, 65, 4, 2, 64) == 0
    assert size(-1, 5, 4, 2, 64) == 0


def test_block_arguments(lib):
    for name in ("qkv", "conv_w", "conv_state", "alpha", "b", "dt", "a", "z", "norm_w", "state", "out",
                 "tape", "ws"):
        assert block(lib, **{name: None}) == NULL
    for name in ("qkv", "conv_w", "conv_state", "z", "norm_w", "state", "out", "tape", "ws"):
        assert block(lib, **{name: MIS}) == ALIGN
    for name in ("qkv", "conv_state", "state", "accepted", "tape"):
        assert commit(lib, **{name: None}) == NULL
    assert commit(lib, state=MIS) == ALIGN
    assert commit(lib, tape=MIS) == ALIGN
    for call in (block, commit):
        assert call(lib, hk=3) == SHAPE
        assert call(lib, hk=0) == SHAPE
        assert call(lib, s=48) == SHAPE
        assert call(lib, s=96) == UNSUP
        assert call(lib, kernel=1) == SHAPE
        assert call(lib, kernel=9) == SHAPE
        assert call(lib, n=65536, pool=65536) == UNSUP
        need = lib.gdn_block_tree_tape_size(2, 5, 2, 4, 64)
        assert need > 0 and call(lib, tape_bytes=need - 1) == SHAPE
    need = lib.gdn_block_tree_workspace_size(2, 5, 2, 4, 64)
    assert need > 0 and block(lib, ws_bytes=need - 1) == SHAPE
    for size in (lib.gdn_block_tree_tape_size, lib.gdn_block_tree_workspace_size):
        assert size(-1, 5, 2, 4, 64) == size(2, 0, 2, 4, 64) == size(2, 65, 2, 4, 64) == 0
        assert size(2, 5, 3, 4, 64) == size(2, 5, 2, 4, 60) == 0


def test_accept_arguments(lib):
    for name in ("tokens", "sampled", "accepted", "n_kept", "next_tokens", "pages", "table", "lens",
                 "new_lens"):
        assert accept(lib, **{name: None}) == NULL
    assert accept(lib, planes=-1) == SHAPE
    assert accept(lib, planes=0, lens=None) == NULL      # new_lens without lengths
    assert accept(lib, planes=0, new_lens=None) == NULL
    assert accept(lib, ps=0) == SHAPE
    assert accept(lib, ps=24) == UNSUP
    assert accept(lib, max_pages=0) == SHAPE
    assert accept(lib, max_pages=1 << 30) == UNSUP
    assert accept(lib, hkv=0) == SHAPE
    assert accept(lib, n_pages=0) == SHAPE
    assert accept(lib, pb=0) == SHAPE
    assert accept(lib, pb=4096 + 16) == SHAPE            # no whole rows
    assert accept(lib, pages=MIS) == ALIGN


def test_sample_arguments(lib):
    for name in ("logits", "u", "tokens"):
        assert sample(lib, **{name: None}) == NULL
    assert sample(lib, rows=-1) == SHAPE
    assert sample(lib, vocab=0) == SHAPE
    assert sample(lib, stride=99) == SHAPE
    assert sample(lib, per_set=0) == SHAPE
    assert sample(lib, dtype=3) == UNSUP
    assert sample(lib, vocab=(1 << 20) + 1) == UNSUP
    assert sample(lib, logits=P + 2) == ALIGN            # fp32 at half a value
    assert sample(lib, rows=0) == OK


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_sample(x, x[:, 0], i, 2, 8, stream=0)
    with pytest.raises(TypeError):
        gdn.gdn_sample(i, x, i, 2, 8, stream=0)
    with pytest.raises(ValueError):
        gdn.gdn_tree_accept(i, i, i, i, i, i, i, None, 1, 2, stream=0)
    with pytest.raises(ValueError):
        gdn.gdn_block_tree_commit(x, x, x, i, i, 1, 2, 1, 1, 32, 4, x, stream=0)
    with pytest.raises(ValueError):
        gdn.gdn_attn_tree(x, x, x, i, i, x, i, 1, 2, 1, 1, 64, 16, 1, 1, 0, 0, 1.0, x, stream=0)


def test_pools_of_a_terabyte(lib):
    assert block(lib, s=128, pool=1 << 22, h=4, slots=P) == UNSUP
    assert block(lib, s=128, pool=1 << 22, h=4, slots=P, n=0) == UNSUP
