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


# 2^256 / (2 pi), and inverse frequencies (bits) with positions that come within 2 units of 2^-32 turn
# of a quarter turn: the small one of cosine and sine shows the angle's own error.
INV_2PI = 0x28be60db9391054a7f09d5f47d4d377036d8a5664f10e4107f9458eaf7aef158
NEAR_QUARTERS = [
    (0x3f4347d4, 2122934198), (0x3f21d5e2, 2040872170), (0x3f7b7378, 2076569594), (0x3f5b0e24, 2045508788),
    (0x3f41b950, 2039619361), (0x3f2e3b52, 2096071377), (0x3f71b182, 2131501801), (0x3f14470a, 2081693231),
    (0x3f013e3b, 2092000254), (0x3f6dd34c, 2056101290), (0x3f5c0c2e, 2145003625), (0x3f7fe5c3, 2131542241),
    (0x3f6e9700, 2117353440), (0x3f4f42f5, 2057640967), (0x3f59a57d, 2064191376), (0x3f765a8f, 2083182781),
    (0x3f696ed8, 2038087938), (0x3f5c7fde, 2135341770), (0x3f599147, 2022093181), (0x3f702ca0, 2052251297),
    (0x3f0f168a, 2116037525), (0x3f43a4bf, 2025415655), (0x3f4d1865, 2090526301), (0x3f5c0c2e, 2034278808),
]


def test_angles_to_a_2_32nd_of_a_turn(lib):
    """Heads of ones and zeros give cosines and sines themselves, rounded once to bf16."""
    n, pairs = len(NEAR_QUARTERS), 32
    bits = [b for b, _ in NEAR_QUARTERS] + [0x3F800000] * (pairs - n)
    pos = [p for _, p in NEAR_QUARTERS] + [-p for _, p in NEAR_QUARTERS] + [2 ** 31 - 1, -2 ** 31]
    for il in (False, True):
        q = torch.zeros(len(pos), 1, 2 * pairs, dtype=torch.bfloat16, device="cuda")
        a, b = (slice(0, None, 2), slice(1, None, 2)) if il else (slice(0, pairs), slice(pairs, None))
        q[:, :, a] = 1
        out = torch.empty_like(q)
        inv = torch.from_numpy(np.array(bits, np.uint32).view(np.float32).copy()).cuda()
        lib.idx_norm_rope(lib.make_norm_rope(q, q_out=out, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), inv_freq=inv,
                                             interleaved=il, q_norm=lib.IDX_NORM_NONE))
        got = out[:, 0].double().cpu().numpy()
        want = np.zeros((len(pos), 2, pairs))
        for i, u in enumerate(bits):
            m, down = (u & 0x7FFFFF) | 0x800000, 150 - (u >> 23)        # the frequency is m 2^-down
            unit = 1 << (256 + down)
            for r, p in enumerate(pos):
                turn = m * INV_2PI * p % unit
                quarter = (4 * turn + unit // 2) // unit
                rest = float((4 * turn - quarter * unit) / unit) * np.pi / 2
                c, s = np.cos(rest), np.sin(rest)
                want[r, :, i] = [(c, s), (-s, c), (-c, -s), (s, -c)][quarter % 4]
        got = np.stack([got[:, a], got[:, b]], 1)
        assert (np.abs(got - want) <= 2 * np.pi * 2.0 ** -32 + (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "bf16 keys", "e4m3 keys"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_halves_into_the_cache(lib, kv, D, layout):
    """Pairs by halves, heads that turn whole, in part and not at all, into every kind of cache."""
    for R, Hq, Hkv, rot in ((1, 8, 1, D), (70, 5, 3, D // 2), (33, 2, 2, 16), (131, 0, 16, 0)):
        c = Case(lib, R, Hq, Hkv, D, kv, 1, 2, rot, False, seed=R, layout=layout)
        K0, V0 = c.K.clone(), None if c.V is None else c.V.clone()
        ks0, vs0 = [None if s is None else s.clone() for s in (c.ks, c.vs)]
        lib.idx_norm_rope(c.plan())
        c.check()
        page, off = c.slot.long() // PAGE, c.slot.long() % PAGE
        if V0 is not None:
            spare = [x.clone() if x is not None else None for x in (K0, V0, ks0, vs0)]
            lib.idx_write_kv(lib.make_kv_cache(*spare), c.v, c.v, c.slot)
            assert torch.equal(c.V, spare[1]) and (vs0 is None or torch.equal(c.vs, spare[3]))
        K0[page, off] = c.K[page, off]          # nothing else is touched
        assert torch.equal(K0, c.K)
        if ks0 is not None:
            ks0[page, :, off] = c.ks[page, :, off]
            assert torch.equal(ks0, c.ks)
