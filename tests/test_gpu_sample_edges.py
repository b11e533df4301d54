"""idx_sample where its integer arithmetic shows, against tests/test_gpu_sample.py's 64-bit reference."""
import numpy as np
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


@pytest.mark.parametrize("parity", [0, 1])
@pytest.mark.parametrize("V,sigma", [(20000, 1.5), (150000, 3.0), (1500, 4.0)])
def test_borders_at_every_edge(lib, V, sigma, parity):
    """p Z within an fp32 rounding of the mass above an edge of a bin of a 64th of an octave: edges between
    two bins that one thread looks at, and between those of neighbours."""
    rng = np.random.default_rng(V + parity)
    row = (rng.standard_normal(V) * sigma).astype(np.float32)
    x = np.sort(row.astype(np.float64))[::-1]
    w = np.exp(x - x[0])
    below = np.ceil(x[0] * np.log2(np.e)) * 64 - np.rint(64 * x * np.log2(np.e))
    cum = np.cumsum(w) / w.sum()
    code = below.astype(int) + 63
    edges = np.flatnonzero((np.diff(code) != 0) & (code[1:] % 2 == parity))
    edges = edges[(cum[edges] > 0.01) & (cum[edges] < 0.995)]
    assert edges.size >= 30
    p = cum[edges][rng.permutation(edges.size)[:120]].astype(np.float32)
    p = np.concatenate([p, np.nextafter(p, np.float32(0)), np.nextafter(p, np.float32(1))])
    many = torch.from_numpy(row).cuda().expand(p.size, V).contiguous()
    check(lib, many, rng.random(p.size), top_p=p)
    few = slice(0, p.size, 7)
    check(lib, many[few].contiguous(), rng.random(p[few].size), top_p=p[few], min_p=np.full(p[few].size, 1e-3))


def _near_borders(rng, ref_zero, n):
    """n pairs of logits (the lighter first) and temperatures, and a u on either side of the lighter one's
    share, as near as the weights' own error allows: 2 in 2^36.2 and a unit of 2^-43 of the heavier at most."""
    got = []
    while len(got) < n:
        T = np.exp(rng.uniform(-3, 3, 1 << 18)).astype(np.float32)
        top = rng.uniform(-80, 80, T.size) * T if ref_zero else np.sign(rng.uniform(-1, 1, T.size)) * rng.uniform(100, 3000, T.size) * T
        top = top.astype(np.float32)
        low = (top - rng.uniform(0, 8, T.size) * T).astype(np.float32)
        d = (top.astype(np.float64) - low) / T
        share = 1 / (1 + np.exp(d))                      # off by 2^-49 of itself at most
        u = share.astype(np.float32)
        away = (u - share) / share
        least = 2.0 ** -35 + np.exp2(d * np.log2(np.e) - 43)
        for i in np.flatnonzero((np.abs(away) > least) & (np.abs(away) < 4 * least) & (low < top)):
            got.append((low[i], top[i], T[i], u[i], away[i] < 0))
    return got[:n]


@pytest.mark.parametrize("ref_zero", [True, False])
@pytest.mark.parametrize("V", [2, 40, 5000])
def test_weights_to_a_2_35th(lib, V, ref_zero):
    """The lighter of two tokens is drawn for u just below its share and not just above: by the whole row,
    by a list and by what top-p sums."""
    rng = np.random.default_rng(V + ref_zero)
    n = 400
    low, top, T, u, lighter = (np.array(v) for v in zip(*_near_borders(rng, ref_zero, n)))
    assert 0.3 < lighter.mean() < 0.7
    at = np.sort(np.stack([rng.permutation(V)[:2] for _ in range(n)]), 1)
    x = np.full((n, V), -np.inf, np.float32)
    r = np.arange(n)
    x[r, at[:, 0]], x[r, at[:, 1]] = low, top
    want = np.where(lighter, at[:, 0], at[:, 1])
    x = torch.from_numpy(x).cuda()
    for kw in (dict(), dict(top_p=np.full(n, 1 - 2.0 ** -24)), dict(top_k=np.full(n, 2)), dict(min_p=np.full(n, 2.0 ** -20))):
        token, _ = run(lib, x, u, temperature=T, **kw)
        assert (token == want).all(), (kw.keys(), np.flatnonzero(token != want).size)
