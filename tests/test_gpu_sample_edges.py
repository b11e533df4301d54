"""idx_sample where its integer arithmetic shows, against tests/test_gpu_sample.py's 64-bit reference."""
import pytest
import torch

from tests.test_gpu_sample import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


@pytest.mark.parametrize("kw", [dict(), dict(top_k=[3] * 5), dict(top_p=[1 - 2.0 ** -24] * 5)])
def test_numbers_of_one_and_above_are_the_last_below_one(lib, kw):
    """u = 1 draws what 1 - 2^-24 draws, also where the last tokens weigh less than 2^-24 together."""
    x = torch.full((5, 700), -float("inf"), device="cuda")
    x[:, 3] = 0.0
    x[:, 600] = -18.0      # 2^-26 of the first
    x[:, 699] = -21.0
    check(lib, x, [1.0, 1 - 2.0 ** -24, 1.5, float("inf"), 3e38], **kw)
    token, _ = run(lib, x, [1.0] * 5, **kw)
    assert (token == 3).all()
