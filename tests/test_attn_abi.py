"""Host-side refusals of the attention layer's calls (no GPU needed): every bad argument gives
its documented status before anything is enqueued, and calls with nothing to do are no-ops."""
import pytest

import gated_deltanet_linear_scan_gb300 as gdn

OK, NULL, SHAPE, UNSUP, ALIGN = 0, 1, 2, 3, 4
P, MIS = 0x10000, 0x10004  # fake device addresses, aligned and not; never dereferenced here
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    gdn.build_if_needed()
    return gdn.library()


def append(lib, k=P, v=P, kp=P, vp=P, table=P, lens=P, cu=P, n=2, total=6, hkv=2, d=64, ps=16,
           n_pages=8, max_pages=4, ks=None, vs=None, dtype=2, slots=None, pool=2):
    return lib.gdn_kv_append(k, v, kp, vp, table, lens, cu, n, total, hkv, d, ps, n_pages,
                             max_pages, hkv * d if ks is None else ks, hkv * d if vs is None else vs,
                             dtype, slots, pool, None, None)


def decode(lib, q=P, kp=P, vp=P, table=P, lens=P, out=P, n=2, tokens=1, hq=4, hkv=2, d=64, ps=16,
           n_pages=8, max_pages=4, window=0, sinks=0, qs=None, dtype=2, slots=None, pool=2, ws=P,
           ws_bytes=BIG):
    return lib.gdn_attn_decode(q, kp, vp, table, lens, out, n, tokens, hq, hkv, d, ps, n_pages,
                               max_pages, window, sinks, 0.1, hq * d if qs is None else qs, dtype,
                               slots, pool, None, ws, ws_bytes, None)


def prefill(lib, q=P, kp=P, vp=P, table=P, lens=P, out=P, cu=P, n=2, total=6, longest=4, hq=4,
            hkv=2, d=64, ps=16, n_pages=8, max_pages=4, window=0, sinks=0, qs=None, dtype=2,
            slots=None, pool=2, ws=P, ws_bytes=BIG):
    return lib.gdn_attn_prefill(q, kp, vp, table, lens, out, cu, n, total, longest, hq, hkv, d, ps,
                                n_pages, max_pages, window, sinks, 0.1,
                                hq * d if qs is None else qs, dtype, slots, pool, None, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("call", [append, decode, prefill])
def test_cache_arguments(lib, call):
    for name in ("kp", "vp", "table", "lens"):
        assert call(lib, **{name: None}) == NULL
    assert call(lib, n=-1) == SHAPE
    assert call(lib, hkv=0) == SHAPE
    assert call(lib, n_pages=0) == SHAPE
    assert call(lib, max_pages=0) == SHAPE
    assert call(lib, ps=0) == SHAPE
    assert call(lib, ps=24) == UNSUP
    assert call(lib, ps=4) == UNSUP
    assert call(lib, ps=512) == UNSUP
    assert call(lib, d=96) == UNSUP
    assert call(lib, dtype=3) == UNSUP
    assert call(lib, dtype=-1) == UNSUP
    assert call(lib, n_pages=1 << 30) == UNSUP       # rows past 32 bits
    assert call(lib, max_pages=1 << 30) == UNSUP     # positions past 32 bits
    assert call(lib, pool=1) == SHAPE                # no slots and pool < n_seqs
    assert call(lib, slots=P, pool=0) == SHAPE
    assert call(lib, kp=MIS) == ALIGN
    assert call(lib, vp=MIS) == ALIGN
    assert call(lib, n=0) == OK


def test_append_arguments(lib):
    assert append(lib, k=None) == NULL
    assert append(lib, v=None) == NULL
    assert append(lib, total=-1) == SHAPE
    assert append(lib, cu=None, total=5) == SHAPE    # five rows over two sequences
    assert append(lib, ks=127) == SHAPE              # rows overlap
    assert append(lib, vs=132) == ALIGN              # rows not 16-byte aligned
    assert append(lib, k=MIS) == ALIGN
    assert append(lib, total=0) == OK


def test_decode_arguments(lib):
    assert decode(lib, q=None) == NULL
    assert decode(lib, out=None) == NULL
    assert decode(lib, ws=None) == NULL
    assert decode(lib, tokens=0) == SHAPE
    assert decode(lib, tokens=65) == UNSUP
    assert decode(lib, hq=5) == SHAPE                # not a multiple of the key heads
    assert decode(lib, hq=0) == SHAPE
    assert decode(lib, window=-1) == SHAPE
    assert decode(lib, sinks=-1) == SHAPE
    assert decode(lib, qs=255) == SHAPE
    assert decode(lib, qs=260) == ALIGN
    assert decode(lib, q=MIS) == ALIGN
    assert decode(lib, out=MIS) == ALIGN
    assert decode(lib, ws=MIS) == ALIGN
    need = lib.gdn_attn_decode_workspace_size(2, 1, 4, 2, 64)
    assert need > 0 and decode(lib, ws_bytes=need - 1) == SHAPE
    assert lib.gdn_attn_decode_workspace_size(2, 1, 5, 2, 64) == 0
    assert lib.gdn_attn_decode_workspace_size(2, 1, 4, 2, 48) == 0
    assert lib.gdn_attn_decode_workspace_size(2, 0, 4, 2, 64) == 0


def test_prefill_arguments(lib):
    assert prefill(lib, q=None) == NULL
    assert prefill(lib, out=None) == NULL
    assert prefill(lib, cu=None) == NULL
    assert prefill(lib, total=-1) == SHAPE
    assert prefill(lib, longest=-1) == SHAPE
    assert prefill(lib, hq=5) == SHAPE
    assert prefill(lib, window=-1) == SHAPE
    assert prefill(lib, sinks=-1) == SHAPE
    assert prefill(lib, qs=255) == SHAPE
    assert prefill(lib, qs=260) == ALIGN
    assert prefill(lib, q=MIS) == ALIGN
    assert prefill(lib, out=MIS) == ALIGN
    assert prefill(lib, total=0) == OK
    assert lib.gdn_attn_prefill_workspace_size(2, 6, 5, 2, 64) == 0


def test_pages_arguments(lib):
    def reserve(pages=P, table=P, lens=P, refs=P, new=P, n=2, ps=16, planes=2, n_pages=8, pb=64,
                max_pages=4, slots=None, pool=2, ws=P, ws_bytes=BIG):
        return lib.gdn_pages_reserve(pages, table, lens, refs, new, n, ps, planes, n_pages, pb,
                                     max_pages, slots, pool, None, ws, ws_bytes, None)

    def fork(pages=P, table=P, lens=P, refs=P, parents=P, children=P, n=2, ps=16, planes=2,
             n_pages=8, pb=64, max_pages=4, pool=2, ws=P, ws_bytes=BIG):
        return lib.gdn_pages_fork(pages, table, lens, refs, parents, children, n, ps, planes,
                                  n_pages, pb, max_pages, pool, None, ws, ws_bytes, None)

    def compact(pages=P, table=P, lens=P, refs=P, ps=16, planes=2, n_pages=8, pb=64, max_pages=4,
                pool=2, ws=P, ws_bytes=BIG):
        return lib.gdn_pages_compact(pages, table, lens, refs, ps, planes, n_pages, pb, max_pages,
                                     pool, None, ws, ws_bytes, None)

    def truncate(table=P, lens=P, refs=P, new=P, n=2, ps=16, n_pages=8, max_pages=4, slots=None,
                 pool=2):
        return lib.gdn_pages_truncate(table, lens, refs, new, n, ps, n_pages, max_pages, slots,
                                      pool, None, None)

    for f in (reserve, fork, compact, truncate):
        for name in ("table", "lens", "refs"):
            assert f(**{name: None}) == NULL
        assert f(ps=0) == SHAPE
        assert f(ps=48) == UNSUP
        assert f(n_pages=0) == SHAPE
        assert f(max_pages=0) == SHAPE
        assert f(max_pages=1 << 30) == UNSUP
        assert f(pool=0) == SHAPE
    for f in (reserve, fork, compact):
        assert f(pages=None) == NULL
        assert f(pages=MIS) == ALIGN
        assert f(planes=0) == SHAPE
        assert f(pb=24) == SHAPE
        assert f(ws=None) == NULL
        assert f(ws=MIS) == ALIGN
        assert f(ws_bytes=lib.gdn_pages_workspace_size(0, 8) - 1) == SHAPE
    assert reserve(new=None) == NULL
    assert reserve(n=-1) == SHAPE
    assert reserve(pool=1) == SHAPE
    assert reserve(n=0) == OK
    assert fork(parents=None) == NULL
    assert fork(children=None) == NULL
    assert fork(n=-1) == SHAPE
    assert fork(n=0) == OK
    assert truncate(n=-1) == SHAPE
    assert truncate(n=0) == OK
    copy = lib.gdn_pages_copy
    assert copy(P, None, P, 1, 1, 1, 16, None, None) == NULL
    assert copy(None, P, P, 1, 1, 1, 16, None, None) == NULL
    assert copy(P, P, P, -1, 1, 1, 16, None, None) == SHAPE
    assert copy(P, P, P, 1, 1, 1, 8, None, None) == SHAPE
    assert copy(MIS, P, P, 1, 1, 1, 16, None, None) == ALIGN
    assert copy(P, P, P, 0, 1, 1, 16, None, None) == OK
    assert lib.gdn_pages_workspace_size(-1, 8) == 0
    assert lib.gdn_pages_workspace_size(1, 0) == 0


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(x, x, x, x, x, x, None, 2, 2, 4, 64, 16, 1, 1, stream=0)
    with pytest.raises(TypeError):
        gdn._dtype(torch.zeros(1, dtype=torch.int32), "k_pages")


def test_decode_workspace_does_not_depend_on_the_batch(lib):
    """Partial results are one pair per CTA of the grid, however long the batch."""
    a = lib.gdn_attn_decode_workspace_size(1, 1, 4, 2, 128)
    assert a == lib.gdn_attn_decode_workspace_size(512, 4, 64, 8, 128) > 0
