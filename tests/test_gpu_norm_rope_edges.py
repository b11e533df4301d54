"""idx_norm_rope at the ends of its ranges, against the formulas of include/idx.h."""
import pytest
import torch

from tests.test_gpu_norm_rope import Case

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
