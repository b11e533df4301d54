"""idx_tree_tables and idx_write_kv where their inputs leave the usual: no rows asked for, and
NaN and infinities among the values."""
import numpy as np
import pytest
import torch

from tests.test_gpu_tree_tables import PAGE, Tables, _codes

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


@pytest.mark.parametrize("D", [64, 128])
def test_written_nan_and_infinity(lib, D):
    """E4M3: a NaN is left out of its vector's amax and becomes a NaN code; a vector of NaN gets
    scale 1; an infinity makes the scale infinite and takes the vector.  bf16: as given."""
    x = torch.randn(4, 2, D, device="cuda").bfloat16()
    x[0, 0, 3] = x[1, 1, D - 1] = float("nan")
    x[1, 1, 0] = -100.0
    x[2, 0] = float("nan")
    x[3, 1, 5] = float("-inf")
    k, v = (torch.zeros(1, PAGE, 2, D, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(1, 2, PAGE, device="cuda") for _ in "kv")
    slot = torch.arange(4, dtype=torch.int32, device="cuda")
    lib.idx_write_kv(lib.make_kv_cache(k, v, ks, vs), x, x, slot)
    f = x.float().cpu().numpy()
    nan = np.isnan(f)
    clean = np.where(nan, 0, f).astype(np.float32)
    want, scale = _codes(np.where(np.isinf(clean), 0, clean))
    scale[2, 0], scale[3, 1], want[3, 1] = 1.0, np.inf, np.where(np.signbit(f[3, 1]), 128, 0)
    nan[3, 1, 5] = True
    for codes, sc in ((k, ks), (v, vs)):
        got = codes[0, :4].cpu().numpy()
        assert ((got[nan] & 127) == 127).all()
        assert np.array_equal(got[~nan], want[~nan])
        assert np.array_equal(sc[0, :, :4].cpu().numpy().T, scale)
    kb, vb = (torch.zeros(1, PAGE, 2, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lib.idx_write_kv(lib.make_kv_cache(kb, vb), x, x, slot)
    assert torch.equal(kb[0, :4].view(torch.int16), x.view(torch.int16)) and torch.equal(vb.view(torch.int16), kb.view(torch.int16))
