"""The calls of a verify step together, and what single calls' tests leave out: every pair of
significands through the E4M3 quotient, caches without a common row pitch, states used again."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import tree_util as tu
from tests.test_gpu_tree_attention import _select, _trees

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def test_the_example_step(lib):
    spec = importlib.util.spec_from_file_location("tree_step", os.path.join(ROOT, "examples", "tree_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    g = mod.main(verbose=False)
    s, R = g["step"], g["R"]
    slots = s.slot[:R]
    assert bool((slots >= 0).all()) and slots.unique().numel() == R
    # requests whose cached positions are all selected: the dense call sees the same set.  Both
    # outputs are within 2^-8 |o| + 2^-8 max |v| of the exact one (roundings of the output and
    # of the probabilities, with room for the scores' 2^-16).
    dense, lse = torch.empty_like(g["out"]), torch.empty_like(g["lse"])
    lib.idx_tree_attention(g["problem"], dense, lib.alloc_state(lib.tree_state_size(g["problem"])), lse=lse)
    vmax = float((s.v.view(torch.float8_e4m3fn).float().abs().amax(-1).transpose(1, 2) * s.v_scale).max())
    some = 0
    for i, ctx in enumerate(g["prompts"]):
        a, b = sum(g["new"][:i]), sum(g["new"][:i + 1])
        if ctx > mod.K:
            assert bool((g["sel"][a:b] >= 0).all())
            continue
        some += 1
        d = (g["out"][a:b].double() - dense[a:b].double()).abs()
        assert bool((d <= 2 * (2.0 ** -8 * dense[a:b].double().abs() + 2.0 ** -8 * vmax)).all())
    assert some >= 2
    assert torch.equal(g["token"].long(), g["logits"].argmax(1))


def test_every_quotient_of_bf16_significands(lib):
    """x / (amax / 448) in fp32, to the nearest E4M3 code, for all pairs of significands and
    exponents down to where the quotient vanishes; large and small scales as well."""
    sig = 1.0 + np.arange(128) / 128.0
    rows = []
    for scale in (0, 60, -60, -110, 120, -125):
        for down in (1, 2, 5, 9, 14, 17):
            for i, m in enumerate(sig):
                v = np.concatenate([[m], sig[1:] * 2.0 ** -down])
                v[1::2] *= -1.0
                rows.append(v * 2.0 ** scale)
    x = torch.tensor(np.array(rows), dtype=torch.float32).bfloat16()
    R = x.shape[0]
    x = x.view(R, 1, 128).cuda()
    P = (R + 63) // 64
    k, v = (torch.zeros(P, 64, 1, 128, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(P, 1, 64, device="cuda") for _ in "kv")
    slot = torch.arange(R, dtype=torch.int32, device="cuda")
    lib.idx_write_kv(lib.make_kv_cache(k, v, ks, vs), x, x, slot)
    f = x.float().cpu().numpy()[:, 0]
    sc = (np.abs(f).max(1) / np.float32(448.0)).astype(np.float32)
    want = torch.from_numpy((f / sc[:, None]).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for codes, scales in ((k, ks), (v, vs)):
        assert torch.equal(codes.view(-1, 128)[:R].cpu(), want)
        assert np.array_equal(scales.view(-1)[:R].cpu().numpy(), sc)


def _uneven(step, kv):
    """The step's cache moved to strides without a common pitch of a row."""
    P, H, D = step.P, step.Hkv, step.D
    unit = 16 if kv == "e4m3" else 8
    token = H * D + unit
    page = 64 * token + 3 * unit
    moved = []
    for x in (step.k, step.v):
        raw = torch.zeros(P * page, dtype=x.dtype, device="cuda")
        y = raw.as_strided((P, 64, H, D), (page, token, D, 1))
        y.copy_(x)
        moved.append(y)
    step.k, step.v = moved
    step.cache = step.lib.make_kv_cache(step.k, step.v, step.k_scale, step.v_scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [8, 64, 256])
def test_strides_without_a_common_pitch(lib, kv, D, Hq):
    ctx, new = [0, 70, 900], [3, 4, 9]
    s = tu.Step(ctx, new, Hq, 2, D, kv, masks=_trees(40, new), seed=41)
    _uneven(s, kv)
    out, lse = s.attend()
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse)
    sel = _select(s, 300, 42)
    out, lse = s.attend(sel)
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse, sel)


@pytest.mark.parametrize("Hq,new", [(16, [4]), (128, [20]), (16, [1, 2, 3, 4])])
def test_a_state_serves_call_after_call(lib, Hq, new):
    """Split items leave their counters at zero: equal calls on one state give equal bits."""
    s = tu.Step([20000] * len(new), new, Hq, 2, 128, masks=_trees(43, new), seed=44)
    out, lse = s.attend()
    for _ in range(3):
        again, lse2 = s.attend(state=s.state)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert s.status() == lib.IDX_OK
    # another problem of the same size on the state
    t = tu.Step([15000] * len(new), new, Hq, 2, 128, masks=_trees(45, new), seed=46)
    o, z = t.attend(state=s.state)
    fresh, zf = t.attend()
    assert torch.equal(o, fresh) and torch.equal(z, zf)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [4, 32, 64, 128])
def test_selected_shares_of_many_tiles(lib, kv, D, G):
    """Enough rows for every CTA to walk several tiles and items: each ring of stages turns over."""
    ctx, new = [3579, 700, 2100, 64], [30, 40, 13, 25]
    s = tu.Step(ctx, new, G, 1, D, kv, masks=_trees(47, new), seed=48)
    sel = _select(s, 2048, 49, False)
    out, lse = s.attend(sel)
    assert s.status() == lib.IDX_OK
    tu.check(s, out, lse, sel)
    again, _ = s.attend(sel, state=s.state)
    assert torch.equal(out, again)
