"""idx_tree_attention and idx_tree_attention_selected against the 64-bit reference:
types, head layouts, cache orders, lengths around a page's and a tile's edges, masks
that leave rows empty, stale and masked NaN, long caches, streams, refusals."""
import numpy as np
import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def _trees(seed, new):
    rng = np.random.default_rng(seed)
    return sum((tu.ancestor_masks(tu.random_tree(rng, n)) for n in new), [])


HEADS = [(8, 8), (16, 2), (64, 1), (24, 4), (12, 12), (128, 1), (3, 1)]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["token", "head", "pair"])
def test_ragged_requests(lib, kv, D, layout):
    ctx = [0, 1, 62, 63, 64, 65, 127, 128, 129, 500, 0, 1000]
    new = [1, 1, 3, 1, 4, 7, 2, 64, 5, 0, 33, 17]
    s = tu.Step(ctx, new, 16, 2, D, kv, layout, masks=_trees(1, new), seed=2, q_pad=24)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_head_layouts(lib, heads, kv):
    ctx, new = [700, 5, 130], [5, 2, 11]
    s = tu.Step(ctx, new, *heads, 128, kv, masks=_trees(3, new), seed=4)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("heads", [(8, 1), (64, 8), (64, 1)])
def test_tree_sizes_without_a_mask_are_chains(lib, T, heads):
    s = tu.Step([300], [T], *heads, 128, seed=T)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)


@pytest.mark.parametrize("kv,D,heads,ctx", [
    ("bf16", 128, (8, 1), 40000), ("e4m3", 128, (64, 8), 33333), ("bf16", 64, (32, 8), 20001), ("e4m3", 64, (4, 4), 70000),
    ("bf16", 128, (64, 1), 25000)])
def test_a_long_cache_split_over_the_device(lib, kv, D, heads, ctx):
    new = [6, 3]
    s = tu.Step([ctx, 77], new, *heads, D, kv, masks=_trees(5, new), seed=6)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_peaked_scores(lib, kv):
    """One key far above the rest, early or late: the running maximum moves by much."""
    s = tu.Step([3000, 3000], [2, 2], 8, 1, 128, kv, seed=7, amp=3.0)
    q = s.q
    for i, j in ((0, 5), (1, 2900)):
        k, _ = s.values(i, np.array([j]), 0)
        q[2 * i:2 * i + 2] = (k[0] * 1.5).bfloat16()
    out, lse = s.attend()
    tu.check(s, out, lse)


def test_masks_that_leave_rows_empty(lib):
    ctx, new = [0, 0, 100, 0], [3, 64, 2, 1]
    masks = [0, 0b010, 0] + [0] * 64 + [0, 0] + [1]
    for sel in (None, 1):
        s = tu.Step(ctx, new, 16, 2, 128, masks=masks, seed=8)
        if sel:
            sel = torch.full((s.R, 9), -1, dtype=torch.int32, device="cuda")
        out, lse = s.attend(sel)
        assert s.status() == lib.IDX_OK
        tu.check(s, out, lse, sel)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [(16, 2), (64, 1)])
def test_masked_tokens_may_hold_anything(lib, kv, heads):
    """NaN and infinities in drafted tokens that a row does not see leave it alone; a
    row that sees them gets them."""
    ctx, new = [190, 64], [9, 64]
    masks = [1 << t for t in range(9)] + [(1 << t) | 1 for t in range(64)]
    s = tu.Step(ctx, new, *heads, 128, kv, masks=masks, seed=9)
    for i, u, what in ((0, 4, "nan"), (1, 13, "nan"), (1, 40, "inf")):
        j = ctx[i] + u
        page, off = int(s.table[i, j // 64]), j % 64
        if kv == "e4m3":
            if what == "nan":
                s.k[page, off] = 0x7F
                s.v[page, off] = 0xFF
            else:
                s.v_scale[page, :, off] = float("inf")
                s.v[page, off] = 0x38       # 1.0
        else:
            s.v[page, off] = float(what)
            if what == "nan":
                s.k[page, off] = float("nan")
    out, lse = s.attend()
    clean = torch.ones(s.R, dtype=torch.bool)
    clean[[4, 9 + 13, 9 + 40]] = False
    ro, rl, to, tl = s.reference()
    assert bool(torch.isfinite(out[clean].float()).all())
    assert bool(((out.double() - ro).abs() <= to)[clean].all())
    assert bool(((lse.double() - rl).abs() <= tl)[clean].all())
    assert bool(torch.isnan(out[[4, 9 + 13]].float()).all())
    assert bool(torch.isinf(out[9 + 40].float()).all())


def test_a_cached_nan_reaches_every_row(lib):
    s = tu.Step([500], [3], 8, 1, 128, seed=10)
    s.v[int(s.table[0, 2]), 7, :, 5] = float("nan")
    out, _ = s.attend()
    assert bool(torch.isnan(out[:, :, 5].float()).all())
    keep = [d for d in range(128) if d != 5]
    assert bool(torch.isfinite(out[:, :, keep].float()).all())


def test_offsets_past_32_bits(lib):
    """The request's pages lie behind 2^31 elements of other pages."""
    s = tu.Step([1000], [3], 16, 8, 128, seed=11, first_page=33000)
    assert s.k.stride(0) * 33000 > 2 ** 31
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)
    sel = torch.randperm(1000, device="cuda")[:301].to(torch.int32).expand(3, 301).contiguous()
    out, lse = s.attend(sel)
    tu.check(s, out, lse, sel)


def _select(s, K, seed, pad=True):
    rng = np.random.default_rng(seed)
    sel = np.full((s.R, K), -1, np.int32)
    for i, c in enumerate(s.ctx):
        for r in range(s.start[i], s.start[i + 1]):
            n = min(K, c)
            if pad and n:
                n = int(rng.integers(0, n + 1))
            sel[r, :n] = rng.permutation(c)[:n]
            if pad and n < K:
                sel[r, n] = c + 1      # past the cached tokens: skipped
                sel[r, n:] = rng.permutation(sel[r, n:])
    return torch.from_numpy(sel).cuda()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["token", "head", "pair"])
@pytest.mark.parametrize("K", [1, 63, 300, 2048])
def test_selected_positions(lib, kv, D, layout, K):
    ctx = [0, 1, 62, 64, 129, 500, 3000, 0]
    new = [1, 1, 3, 4, 7, 0, 5, 33]
    s = tu.Step(ctx, new, 16, 2, D, kv, layout, masks=_trees(12, new), seed=13, q_pad=8)
    for pad in (True, False):
        sel = _select(s, K, 14, pad)
        out, lse = s.attend(sel)
        assert s.status() == lib.IDX_OK
        tu.check(s, out, lse, sel)


@pytest.mark.parametrize("heads", HEADS)
def test_selected_head_layouts(lib, heads):
    ctx, new = [3000, 40], [4, 3]
    s = tu.Step(ctx, new, *heads, 128, "e4m3", seed=15)
    sel = _select(s, 777, 16, False)
    out, lse = s.attend(sel)
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse, sel)


def test_selected_masked_tokens_may_hold_anything(lib):
    s = tu.Step([200], [5], 16, 2, 128, masks=[1 << t for t in range(5)], seed=17)
    j = 200 + 3
    s.v[int(s.table[0, j // 64]), j % 64] = float("nan")
    s.k[int(s.table[0, j // 64]), j % 64] = float("inf")
    sel = _select(s, 100, 18, False)
    out, _ = s.attend(sel)
    assert bool(torch.isfinite(out[[0, 1, 2, 4]].float()).all())
    assert bool(torch.isnan(out[3].float()).all())


def test_equal_calls_give_equal_bits_on_any_stream(lib):
    new = [6, 3, 20]
    s = tu.Step([9000, 77, 4000], new, 16, 2, 128, "e4m3", masks=_trees(19, new), seed=20)
    a = s.attend()
    state = s.state
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = s.problem()
    with torch.cuda.stream(side):
        b = s.attend(problem=p, state=state)
    torch.cuda.current_stream().wait_stream(side)
    c = s.attend(problem=p, state=state)
    for x, y in ((a, b), (a, c)):
        assert torch.equal(x[0].view(torch.int16), y[0].view(torch.int16)) and torch.equal(x[1], y[1])


def test_a_call_in_a_graph_sees_new_lengths(lib):
    """Lengths and tables are device data: a captured call replays with other ones."""
    new = [4, 4]
    s = tu.Step([3000, 2000], new, 16, 2, 128, seed=21)
    p = s.problem()
    out = torch.empty(s.R, 16, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s.R, 16, device="cuda")
    state = lib.alloc_state(lib.tree_state_size(p))
    lib.idx_tree_attention(p, out, state, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.idx_tree_attention(p, out, state, lse=lse)
    for ctx in ([3000, 2000], [1, 1500], [0, 64]):
        s.ctx = ctx
        s.ctx_len.copy_(torch.tensor(ctx, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        tu.check(s, out, lse)


def test_bad_data_is_clamped_and_reported(lib):
    s = tu.Step([300, 200], [4, 4], 16, 2, 128, seed=22)
    good = s.attend()
    assert s.status() == lib.IDX_OK
    # a page id outside the cache: its tokens are left out, the other request is untouched
    keep = int(s.table[0, 1])
    for bad in (-1, s.P, 2 ** 31 - 1):
        s.page_table[0, 1] = bad
        out, lse = s.attend()
        assert s.status() == lib.IDX_EDEVICE
        assert s.status() == lib.IDX_OK          # reading clears it
        assert torch.equal(out[4:], good[0][4:])
        left = tu.Step([300 - 64, 200], [4, 4], 16, 2, 128, seed=22)
        left.k, left.v, left.q = s.k, s.v, s.q
        left.table = np.concatenate([s.table[:, :1], s.table[:, 2:]], 1)
        left.table[1, :] = -1
        left.table[1, :s.table.shape[1]][:1] = s.table[1, 0]
        left.table[1] = np.pad(s.table[1], (0, 0))[:left.table.shape[1]]
        ro, rl, to, tl = left.reference()
        assert bool(((out.double() - ro).abs() <= to)[:4].all())
    s.page_table[0, 1] = keep
    # a context above the host's bound is cut to it
    s.attend(problem=s.problem(max_ctx=250))
    assert s.status() == lib.IDX_EDEVICE
    # more rows than the host's bound: the rest are not written
    out, _ = s.attend(problem=s.problem(max_new=3))
    assert s.status() == lib.IDX_EDEVICE
    assert bool((out[3] == 7).all())


def test_refusals(lib):
    s = tu.Step([300], [4], 16, 2, 128, seed=23)
    sel = _select(s, 10, 24)
    out = torch.empty(4, 16, 128, dtype=torch.bfloat16, device="cuda")
    p = s.problem()
    state = lib.alloc_state(lib.tree_state_size(p, 10))
    for kw in (dict(q=None), dict(page_table=None), dict(R=0), dict(Q=0), dict(Hq=15), dict(max_ctx=-1), dict(max_new=0),
               dict(scale=float("nan")), dict(q_row_stride=16 * 128 - 8), dict(q_row_stride=16 * 128 + 1),
               dict(max_ctx=64 * 64 * 1000)):
        with pytest.raises(lib.IdxError) as e:
            lib.lib.idx_tree_attention  # the entry point itself exists
            lib._check(_call(lib, s.problem(**kw), out, state), "idx_tree_attention")
        assert e.value.status == lib.IDX_EINVAL, kw
        assert lib.tree_state_size(s.problem(**kw)) == 0, kw
    for kw in (dict(max_new=65), dict(Q=5000), dict(R=70000)):
        assert _call(lib, s.problem(**kw), out, state) == lib.IDX_EUNSUPPORTED, kw
    assert _call(lib, p, None, state) == lib.IDX_EINVAL
    assert _call(lib, p, out, state[16:]) == lib.IDX_EINVAL          # misaligned
    assert _call(lib, p, out, state[:1]) == lib.IDX_EINVAL           # too small
    with pytest.raises(ValueError):
        lib.idx_tree_attention(p, out[:3], state)
    with pytest.raises(ValueError):
        lib.idx_tree_attention_selected(p, sel[:2], out, state)
    with pytest.raises(lib.IdxError):
        lib.idx_tree_attention_selected(p, torch.zeros(4, 2049, dtype=torch.int32, device="cuda"), out, state)
    many = tu.Step([30], [1], 256, 1, 128, seed=25)
    with pytest.raises(lib.IdxError) as e:
        many.attend(_select(many, 10, 26))
    assert e.value.status == lib.IDX_EUNSUPPORTED
    with pytest.raises(ValueError):
        lib.make_kv_cache(s.k, s.v[:, :, :1])
    with pytest.raises(ValueError):
        lib.make_kv_cache(s.k.float(), s.v.float())
    with pytest.raises(ValueError):
        lib.make_kv_cache(s.k, s.v, torch.ones(s.P, 2, 64, device="cuda"))


def _call(lib, p, out, state):
    import ctypes
    return lib.lib.idx_tree_attention(ctypes.byref(p), lib._ptr(out), None, lib._ptr(state), state.numel(), lib._stream(None))
