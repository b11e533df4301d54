"""Attention where its paths meet their edges: references that rise over a whole cache, scales and
scores at their limits, more requests than a warp or a CTA sums at once."""
import numpy as np
import pytest
import torch

from tests import tree_util as tu
from tests.test_gpu_tree_attention import _select, _trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def _rising(step, i, h, rise):
    """Keys of request i, head h grow by `rise` a page: scores of spread 1 become ones of spread
    rise, 2 rise, 3 rise ..., whose maxima over a page's 64 keys lie some 2.4 rise apart."""
    ctx = step.ctx[i]
    j = np.arange(ctx)
    page = torch.from_numpy(step.table[i, j // 64].astype(np.int64)).cuda()
    off = torch.from_numpy(j % 64).cuda()
    grow = torch.from_numpy(rise * (1.0 + j // 64)).cuda()[:, None]
    if step.kv == "bf16":
        step.k[page, off, h] = (step.k[page, off, h].double() * grow).bfloat16()
    else:
        step.k_scale[page, h, off] = (step.k_scale[page, h, off].double() * grow[:, 0]).float()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,new", [(128, [1]), (64, [64]), (96, [5]), (16, [3])])
def test_references_that_rise_page_after_page(lib, kv, D, Hq, new):
    """Scores that pass their row's reference by 2^30 (21 in natural units) in one page after
    another: O is scaled again and again, each time after the product that wrote it."""
    s = tu.Step([700], new, Hq, 1, D, kv, masks=_trees(50, new), seed=51)
    _rising(s, 0, 0, 12.0)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)
    again, _ = s.attend(state=s.state)
    assert torch.equal(out, again)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,new", [((8, 2), 3), ((32, 1), 1), ((64, 1), 1), ((16, 2), 16)])
def test_many_items_whose_first_key_some_rows_do_not_see(lib, kv, heads, new):
    """Items that begin with a tile every row sees the first key of, and items that do not (no
    cached token), in turn within one CTA's share."""
    ctx = [0, 40, 130, 0, 300, 0, 128, 1] * 25
    rng = np.random.default_rng(52)
    counts = rng.integers(1, new + 1, len(ctx)).tolist()
    s = tu.Step(ctx, counts, *heads, 128, kv, masks=_trees(53, counts), seed=54)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,new", [(16, [3, 2, 4]), (128, [1, 1, 1]), (64, [64, 20, 5])])
def test_a_scale_of_zero_takes_the_mean(lib, kv, D, Hq, new):
    """Scores of 0 for every visible key, whatever the masked ones hold (stale slots are NaN)."""
    s = tu.Step([100, 300, 0], new, Hq, 1, D, kv, masks=_trees(55, new), seed=56)
    s.scale = 0.0
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)
    sel = _select(s, 150, 57)
    out, lse = s.attend(sel)
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse, sel)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,new", [((8, 1), 3), ((32, 1), 1), ((16, 2), 2), ((64, 1), 1), ((128, 1), 2)])
def test_scores_of_minus_infinity_add_nothing(lib, D, heads, new):
    """Whole tiles of visible keys with scores of -infinity, in front of others: exp(-inf) = 0."""
    s = tu.Step([400], [new], *heads, D, seed=60)
    s.q[:, :, 0].abs_().clamp_(min=0.5)
    j = np.arange(256)
    page, off = torch.from_numpy(s.table[0, j // 64].astype(np.int64)).cuda(), torch.from_numpy(j % 64).cuda()
    s.k[page, off, :, 0] = float("-inf")
    rest = torch.arange(256, 400, dtype=torch.int32, device="cuda").expand(new, 144).contiguous()
    ro, rl, to, tl = s.reference(rest)       # the same keys but those
    every = torch.arange(400, dtype=torch.int32, device="cuda").expand(new, 400).contiguous()
    for sel in (None, every):
        out, lse = s.attend(sel)
        assert s.status() == lib.IDX_OK
        assert bool(((out.double() - ro).abs() <= to).all())
        assert bool(((lse.double() - rl).abs() <= tl).all())
    # rows whose every score is -infinity have nothing to weigh
    s.k[:, :, :, 0] = float("-inf")
    for sel in (None, every):
        out, lse = s.attend(sel)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("Q", [33, 64, 384, 400, 641, 1000, 4096])
@pytest.mark.parametrize("kv,heads", [("bf16", (8, 1)), ("e4m3", (16, 2)), ("bf16", (128, 1)), ("e4m3", (96, 1))])
def test_many_requests(lib, kv, heads, Q):
    """More requests than a warp sums (32), than a CTA does in one go (384 to 640), and the most
    there may be; empty ones among them."""
    rng = np.random.default_rng(Q)
    ctx = rng.integers(0, 150, Q)
    new = rng.integers(0, 3, Q)
    for i in (31, 32, 383, 384, 639, 640, Q - 1):      # where a scan's chunks end
        if i < Q:
            ctx[i], new[i] = 130 + i % 7, 1 + i % 2
    if Q > 1000:
        new[rng.random(Q) < 0.7] = 0
    ctx, new = ctx.tolist(), new.tolist()
    s = tu.Step(ctx, new, *heads, 64, kv, masks=_trees(61, new), seed=62)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)
    sel = _select(s, 70, 63)
    out, lse = s.attend(sel)
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse, sel)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Q,ctx,heads,new", [(1, 3000, (8, 1), 2), (16, 600, (16, 16), 2), (1, 3000, (128, 1), 1), (16, 600, (512, 8), 1),
                                             (1, 3000, (64, 1), 4), (8, 600, (512, 8), 5)])
def test_a_cached_nan_reaches_rows_that_hardly_weigh_it(lib, kv, D, Q, ctx, heads, new):
    """A visible V that is NaN, under a probability that vanishes beside a later key's: the
    weight is not zero, so the output is NaN, in whichever share, stream or order they meet."""
    s = tu.Step([ctx] * Q, [new] * Q, *heads, D, kv, seed=64)
    u = torch.randint(0, 2, (D,), device="cuda").double() * 2 - 1
    s.q[:] = u.bfloat16()
    for i in range(Q):
        page, off = int(s.table[i, 0]), 5
        s.v[page, off, :, 7] = 0x7F if kv == "e4m3" else float("nan")
        page, off = int(s.table[i, 300 // 64]), 300 % 64
        if kv == "e4m3":      # scores of 20 sqrt(D) there, against some 2 elsewhere
            s.k[page, off] = u.to(torch.float8_e4m3fn).view(torch.uint8)
            s.k_scale[page, :, off] = 20.0
        else:
            s.k[page, off] = (20.0 * u).bfloat16()
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)
    assert bool(torch.isnan(out[:, :, 7].float()).all())


@pytest.mark.parametrize("Q,Hkv,G,ctx", [(32, 1024, 1, 2 ** 25), (4096, 16, 1, 2 ** 24), (4096, 8, 64, 2 ** 24)])
def test_tiles_past_32_bits_are_reported(lib, Q, Hkv, G, ctx):
    """Requests that share their rows (row_start does not ascend) pass the host's bounds; a launch
    of so many tiles that their count would wrap does nothing."""
    new, tile = 4, 128 if 4 * G <= 32 else 64
    assert 2 ** 32 < Q // 2 * Hkv * ((ctx + new + tile - 1) // tile) < 2 ** 32 + 2 ** 20
    k, v = (torch.zeros(1, 64, Hkv, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q = torch.zeros(new, Hkv * G, 64, dtype=torch.bfloat16, device="cuda")
    row_start = torch.tensor([0, new] * (Q // 2) + [0], dtype=torch.int32, device="cuda")
    table = torch.zeros(Q, ctx // 64 + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((Q,), ctx, dtype=torch.int32, device="cuda")
    p = lib.make_tree_problem(q, lib.make_kv_cache(k, v), table, lens, row_start, None, ctx, new, 0.125)
    out = torch.full((new, Hkv * G, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    state = lib.alloc_state(lib.tree_state_size(p))
    lib.idx_tree_attention(p, out, state)
    assert lib.last_device_status(state) == lib.IDX_EDEVICE
    assert bool((out == 7).all())
