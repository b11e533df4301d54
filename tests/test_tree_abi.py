"""Arguments that the verify step's entry points reject on the host, before any GPU call."""
import ctypes

import pytest

FAKE = 1 << 20     # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def _cache(lib, **kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, P=8, page_stride=64 * 2 * 128, token_stride=2 * 128, head_stride=128,
             Hkv=2, D=128, kv_dtype=lib.IDX_KV_BF16)
    a.update(kw)
    return lib.KvCache(**a)


def _tables(lib, **kw):
    a = {f: FAKE for f in ("ctx_len", "new_len", "free_pages", "free_count", "page_table", "row_start", "row_req", "row_bound",
                           "row_pos", "slot", "mask", "parent")}
    a.update(free_left=FAKE + 64, P=8, Q=2, pt_stride=4, cap=8)
    a.update(kw)
    return lib.TreeTables(**a)


def _problem(lib, cache=None, **kw):
    a = dict(q=FAKE, q_row_stride=16 * 128, cache=cache or _cache(lib), page_table=FAKE, ctx_len=FAKE, row_start=FAKE, mask=FAKE,
             R=8, Q=2, pt_stride=4, max_ctx=256, max_new=8, Hq=16, scale=0.1)
    a.update(kw)
    return lib.TreeProblem(**a)


BAD_CACHE = [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(P=0), dict(page_stride=0), dict(token_stride=-256),
             dict(head_stride=4), dict(Hkv=0), dict(kv_dtype=7), dict(k_scale=FAKE), dict(kv_dtype=0)]
NO_CACHE = [dict(D=96), dict(Hkv=1025), dict(P=2 ** 31 // 64 + 1)]


def test_the_constants(lib):
    assert lib.IDX_KV_E4M3 != 7 and lib.IDX_KV_BF16 != 7


@pytest.mark.parametrize("kw", [dict(ctx_len=None), dict(new_len=None), dict(free_pages=None), dict(free_count=None),
                                dict(page_table=None), dict(row_start=None), dict(free_left=None), dict(free_left=FAKE),
                                dict(row_req=None), dict(slot=None), dict(mask=FAKE + 4), dict(Q=0), dict(P=0),
                                dict(pt_stride=0), dict(cap=-1)])
def test_tables(lib, kw):
    t = _tables(lib, **kw)
    assert lib.lib.idx_tree_tables(ctypes.byref(t), FAKE, 1024, None) == lib.IDX_EINVAL


def test_tables_limits_and_state(lib):
    for kw in (dict(Q=4097), dict(P=2 ** 31 // 64 + 1)):
        t = _tables(lib, **kw)
        assert lib.lib.idx_tree_tables(ctypes.byref(t), FAKE, 1024, None) == lib.IDX_EUNSUPPORTED
    t = _tables(lib)
    assert lib.lib.idx_tree_tables(None, FAKE, 1024, None) == lib.IDX_EINVAL
    for state, size in ((None, 1024), (FAKE + 16, 1024), (FAKE, lib.tree_tables_state_size() - 1)):
        assert lib.lib.idx_tree_tables(ctypes.byref(t), state, size, None) == lib.IDX_EINVAL


def _write(lib, cache, k=FAKE, v=FAKE, stride=2 * 128, slot=FAKE, R=4):
    return lib.lib.idx_write_kv(None if cache is None else ctypes.byref(cache), k, v, stride, slot, R, None)


def test_write(lib):
    for kw in BAD_CACHE:
        if kw != dict(kv_dtype=0) or lib.IDX_KV_E4M3 == 0:      # (E4M3 without scales)
            assert _write(lib, _cache(lib, **kw)) == lib.IDX_EINVAL, kw
    for kw in NO_CACHE:
        assert _write(lib, _cache(lib, **kw)) == lib.IDX_EUNSUPPORTED, kw
    c = _cache(lib)
    for kw in (dict(k=None), dict(v=None), dict(slot=None), dict(k=FAKE + 2), dict(stride=128), dict(stride=260), dict(R=-1)):
        assert _write(lib, c, **kw) == lib.IDX_EINVAL, kw
    assert _write(lib, None) == lib.IDX_EINVAL
    assert _write(lib, c, R=2 ** 31) == lib.IDX_EUNSUPPORTED
    assert _write(lib, c, k=None, v=None, slot=None, R=0) == lib.IDX_OK


def _attend(lib, p, out=FAKE, state=FAKE, size=1 << 40, sel=None, sel_k=0):
    r = None if p is None else ctypes.byref(p)
    if sel_k:
        return lib.lib.idx_tree_attention_selected(r, sel, sel_k, out, None, state, size, None)
    return lib.lib.idx_tree_attention(r, out, None, state, size, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=FAKE + 2), dict(page_table=None), dict(ctx_len=None), dict(row_start=None),
                                dict(R=0), dict(Q=0), dict(pt_stride=0), dict(max_ctx=-1), dict(max_ctx=257), dict(max_new=0),
                                dict(Hq=0), dict(Hq=15), dict(scale=-1.0), dict(scale=float("inf")), dict(q_row_stride=2040),
                                dict(q_row_stride=2052)])
def test_attention(lib, kw):
    p = _problem(lib, **kw)
    assert _attend(lib, p) == lib.IDX_EINVAL
    assert _attend(lib, p, sel=FAKE, sel_k=64) == lib.IDX_EINVAL
    assert lib.tree_state_size(p) == 0


def test_attention_limits_state_and_selection(lib):
    for kw in (dict(R=2 ** 20), dict(Q=4097), dict(max_new=65), dict(Hq=2048, q_row_stride=2048 * 128),
               dict(Hq=512, q_row_stride=512 * 128)):
        assert _attend(lib, _problem(lib, **kw)) == lib.IDX_EUNSUPPORTED, kw
    for kw in NO_CACHE:
        assert _attend(lib, _problem(lib, cache=_cache(lib, **kw))) == lib.IDX_EUNSUPPORTED, kw
    p = _problem(lib)
    size = lib.tree_state_size(p)
    assert size > 0 and lib.tree_state_size(p, 2048) > 0
    for args in (dict(out=None), dict(out=FAKE + 8), dict(state=None), dict(state=FAKE + 512), dict(size=size - 1)):
        assert _attend(lib, p, **args) == lib.IDX_EINVAL, args
    assert _attend(lib, None) == lib.IDX_EINVAL
    assert _attend(lib, p, sel=None, sel_k=64) == lib.IDX_EINVAL
    assert _attend(lib, p, sel=FAKE, sel_k=2049) == lib.IDX_EINVAL
    assert lib.tree_state_size(p, 2049) == 0 and lib.tree_state_size(p, -1) == 0
