"""idx_tree_tables and idx_write_kv where their inputs leave the usual: no rows asked for."""
import numpy as np
import pytest
import torch

from tests.test_gpu_tree_tables import Tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


@pytest.mark.parametrize("with_mask", [False, True])
def test_tables_without_rows(lib, with_mask):
    """cap 0: pages, row_start and free_left alone."""
    ctx, new = [0, 63, 64, 500, 128, 7], [1, 64, 1, 0, 200, 57]
    t = Tables(lib, ctx, new, cap=0, seed=58, with_mask=with_mask)
    lib.idx_tree_tables(t.args, t.state)
    assert lib.last_device_status(t.state) == lib.IDX_OK
    table, _, left, _ = t.expected()
    assert np.array_equal(t.page_table.cpu().numpy(), table)
    assert t.o["row_start"].tolist() == [0] + np.cumsum(new).tolist()
    assert t.o["free_left"].tolist() == [left]


def test_tables_without_rows_count_up_to_31_bits(lib):
    """Lengths are cut to 2^30 - 64 and their sums to 2^31 - 1, which is reported."""
    t = Tables(lib, [0, 0, 0], [5, 5, 5], cap=0, seed=59)
    t.keep[1].fill_(2 ** 31 - 1)
    lib.idx_tree_tables(t.args, t.state)
    assert lib.last_device_status(t.state) == lib.IDX_EDEVICE
    n = 2 ** 30 - 64
    assert t.o["row_start"].tolist() == [0, n, 2 * n, 2 ** 31 - 1]
