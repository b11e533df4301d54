"""idx_norm_rope at the ends of its ranges, against the formulas of include/idx.h."""
import numpy as np
import pytest
import torch

from tests.test_gpu_norm_rope import PAGE, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


@pytest.mark.parametrize("value", [2.0 ** 119, 2.0 ** 122, -1.5 * 2.0 ** 124, 3.3895314e38])
def test_constant_heads_past_the_range(lib, value):
    """A head of equal elements has no variance: LayerNorm gives its bias, however large they are."""
    c = Case(lib, 3, 2, 1, 128, "none", 2, 2, seed=1, rot=0)
    c.q[:, 0] = value
    c.k[1] = value
    lib.idx_norm_rope(c.plan())
    c.check()
    assert bool((c.q_out[:, 0] == c.qb.bfloat16()).all()) and bool((c.k_out[1] == c.kb.bfloat16()).all())


def test_scales_below_the_smallest_number(lib):
    """amax / 448 that fp32 rounds to 0: the smallest scale instead, no 0 / 0 beside it.  A value of a
    few units of 2^-149 is its code times that scale, but for the rounding of the product with the weight."""
    c = Case(lib, 6, 1, 2, 64, "e4m3", 1, 1, seed=2, rot=0)
    c.k[:, :, ::2] = 0
    c.kw[:] = 2.0 ** -146
    lib.idx_norm_rope(c.plan())
    page, off = c.slot.long() // PAGE, c.slot.long() % PAGE
    assert bool((c.ks[page, :, off] == 2.0 ** -149).all())
    z, _ = c.exact(c.k, 1, c.kw, None)
    got = c.K.view(torch.float8_e4m3fn)[page, off].double().cpu().numpy() * 2.0 ** -149
    assert (got[:, :, ::2] == 0).all() and (np.abs(got - z) <= 2.0 ** -149 + 2.0 ** -4 * np.abs(z)).all() and np.abs(got).max() > 0
