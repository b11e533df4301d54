"""Sizes and addresses that the verify step's kernels could not follow are refused on the host,
before any GPU call."""
import ctypes

import pytest

from tests.test_tree_abi import FAKE, _attend, _cache, _problem, _tables, _write

INT32_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def test_rows_are_counted_in_31_bits(lib):
    """A thread stores four rows from r on, r < cap a multiple of four: r + 4 has to fit."""
    for cap in (INT32_MAX - 2, INT32_MAX - 1, INT32_MAX):
        assert (cap - 1) // 4 * 4 + 4 > INT32_MAX
        t = _tables(lib, cap=cap)
        assert lib.lib.idx_tree_tables(ctypes.byref(t), FAKE, 1024, None) == lib.IDX_EUNSUPPORTED, cap
    assert (INT32_MAX - 3 - 1) // 4 * 4 + 4 <= INT32_MAX


def test_positions_are_counted_in_31_bits(lib):
    """A request's keys, and the keys of its last tile, are ctx_len + up to 64 tokens + 127."""
    for max_ctx in ((1 << 30) + 1, INT32_MAX - 128, INT32_MAX):
        p = _problem(lib, cache=_cache(lib, Hkv=1), Hq=8, pt_stride=1 << 25, max_ctx=max_ctx)
        for sel_k in (0, 64):
            assert _attend(lib, p, sel=FAKE, sel_k=sel_k) == lib.IDX_EUNSUPPORTED, max_ctx
            assert lib.tree_state_size(p, sel_k) == 0
    p = _problem(lib, cache=_cache(lib, Hkv=1), Hq=8, pt_stride=1 << 25, max_ctx=1 << 30)
    assert lib.tree_state_size(p) > 0 and lib.tree_state_size(p, 64) > 0


@pytest.mark.parametrize("name", ["ctx_len", "new_len", "free_pages", "free_count", "page_table", "row_start", "free_left",
                                  "row_req", "row_bound", "row_pos", "slot", "parent"])
def test_tables_want_aligned_arrays(lib, name):
    t = _tables(lib, **{name: FAKE + 130})
    assert lib.lib.idx_tree_tables(ctypes.byref(t), FAKE, 1024, None) == lib.IDX_EINVAL


@pytest.mark.parametrize("kw", [dict(page_table=FAKE + 2), dict(ctx_len=FAKE + 1), dict(row_start=FAKE + 2), dict(mask=FAKE + 4)])
def test_attention_wants_aligned_arrays(lib, kw):
    p = _problem(lib, **kw)
    assert _attend(lib, p) == lib.IDX_EINVAL
    assert _attend(lib, p, sel=FAKE, sel_k=64) == lib.IDX_EINVAL
    assert lib.tree_state_size(p) == 0


def test_other_arrays_are_aligned_too(lib):
    p = _problem(lib)
    assert _attend(lib, p, sel=FAKE + 2, sel_k=64) == lib.IDX_EINVAL
    assert lib.lib.idx_tree_attention(ctypes.byref(p), FAKE, FAKE + 2, FAKE, 1 << 40, None) == lib.IDX_EINVAL
    assert _write(lib, _cache(lib), slot=FAKE + 2) == lib.IDX_EINVAL
