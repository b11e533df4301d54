"""idx_sample against the definition in include/idx.h in 64 bits.

A token has to be the reference's: the library's sums are off by about 2^-38 of the row's
weight, so a random u lies that close to a border once in millions of rows.  Where the
inputs put u or p on a border exactly (equal logits), both sides are exact.  logprob is
the sum of -(max l - l) / T and -log1p(Z - 1), both <= 0 and each rounded to fp32 (with log1p
2^-22 of itself), but Z is a sum of at most V weights that are each rounded to an odd multiple of
2^-44 of the power of two at or above the largest.  That unit is 2^-43 of the largest at most, and
no weight is off by more: 2^-21 of itself and V 2^-43."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def reference(x, T=1.0, k=0, p=1.0, m=0.0, u=0.0):
    """(token, logprob) of one row of float64 logits."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf
    if not T > 0 or p <= 0 or k == 1:
        return int(np.argmax(x)), 0.0
    T = min(max(T, 2.0 ** -60), 2.0 ** 60)
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / T))
    order = np.argsort(-x, kind="stable")
    if 0 < k < x.size:
        order = order[:k]
    order = order[w[order] > 0]
    if p < 1:
        s = np.cumsum(w[order])
        order = order[:1 + int((s[:-1] < p * s[-1]).sum())]
    if m > 0:
        order = order[w[order] >= min(m, 1.0)]
    kept = np.sort(order)
    s = np.cumsum(w[kept])
    u = 0.0 if not u > 0 else min(u, 1 - 2.0 ** -24)
    j = int((s <= u * s[-1]).sum())
    return int(kept[j]), float(-np.log1p((s[-1] - w[kept[j]]) / w[kept[j]]))


def run(lib, x, u, stream=None, rows=None, **kw):
    R = x.shape[0]
    dev = {n: torch.tensor(np.asarray(v), dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda")
           for n, v in kw.items() if v is not None}
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    logprob = torch.full((R,), 7.0, device="cuda")
    plan = lib.make_sample(x, torch.tensor(np.asarray(u), dtype=torch.float32, device="cuda"), token, logprob=logprob, rows=rows, **dev)
    lib.idx_sample(plan, stream)
    torch.cuda.synchronize()
    return token.cpu().numpy(), logprob.cpu().numpy()


def check(lib, x, u, **kw):
    token, logprob = run(lib, x, u, **kw)
    host = x.double().cpu().numpy()
    f = lambda n, d: np.asarray(kw[n], np.float32).astype(np.float64) if kw.get(n) is not None else np.full(x.shape[0], d)  # noqa: E731
    T, k, p, m, u = f("temperature", 1.0), f("top_k", 0.0), f("top_p", 1.0), f("min_p", 0.0), np.asarray(u, np.float32).astype(np.float64)
    for r in range(x.shape[0]):
        want, lp = reference(host[r], T[r], int(k[r]), p[r], m[r], u[r])
        assert token[r] == want, (r, token[r], want, T[r], k[r], p[r], m[r], u[r])
        if want < 0:
            assert logprob[r] == -np.inf
        else:
            assert abs(logprob[r] - lp) <= 2.0 ** -21 * abs(lp) + x.shape[1] * 2.0 ** -43, (r, logprob[r], lp)


def _mixed(rng, R):
    """Parameters of a batch of many users."""
    return dict(temperature=np.where(rng.random(R) < 0.1, 0.0, rng.uniform(0.2, 2.0, R)), top_k=np.where(rng.random(R) < 0.3, 0, rng.integers(1, 300, R)),
                top_p=np.where(rng.random(R) < 0.3, 1.0, rng.uniform(0.05, 0.999, R)), min_p=np.where(rng.random(R) < 0.5, 0.0, rng.uniform(0.0, 0.3, R)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 5, 127, 128, 129, 1000, 4099, 16385, 50257, 151552, 360448])
def test_sizes(lib, dtype, V):
    rng = np.random.default_rng(V)
    R = 24 if V < 100000 else 6
    x = torch.from_numpy((rng.standard_normal((R, V)) * rng.uniform(0.5, 6, (R, 1)) + rng.uniform(-20, 20, (R, 1))).astype(np.float32)).cuda().to(dtype)
    u = rng.random(R)
    check(lib, x, u)
    kw = _mixed(rng, R)
    check(lib, x, u, **kw)
    for n in kw:
        check(lib, x, u, **{n: kw[n]})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_logits(lib, dtype):
    """Thresholds inside classes of equals: the first of them by index, however many warps and CTAs they span."""
    rng = np.random.default_rng(5)
    for V in (64, 1000, 40000):
        x = torch.from_numpy(rng.integers(0, 3, (40, V)).astype(np.float32)).cuda().to(dtype)
        u = rng.random(40)
        k = rng.integers(2, V, 40)
        check(lib, x, u, top_k=k)
        check(lib, x, u, top_p=rng.uniform(0.01, 0.999, 40))
        check(lib, x, u, top_k=k, top_p=rng.uniform(0.5, 0.999, 40), temperature=rng.uniform(0.5, 3, 40))
        x[:] = 1.5          # one class
        check(lib, x, u, top_k=k, top_p=rng.uniform(0.5, 0.999, 40))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_flat_rows_and_many_kept(lib, dtype):
    """Borders in bins of thousands of elements: cut finer, or found over the whole row."""
    rng = np.random.default_rng(13)
    V = 150001
    for scale in (0.02, 0.3, 1.0):
        x = torch.from_numpy((rng.standard_normal((6, V)) * scale).astype(np.float32)).cuda().to(dtype)
        u = rng.random(6)
        k = [400, 1500, 5000, 20000, 100000, V - 1]
        p = [0.01, 0.3, 0.6, 0.9, 0.99, 0.9999]
        check(lib, x, u, top_k=k)
        check(lib, x, u, top_p=p)
        check(lib, x, u, top_k=k, top_p=p[::-1], min_p=[0.0, 0.1, 0.5, 0.9, 0.0, 0.99])


def test_exact_borders(lib):
    """u Z and p Z on a border: equal weights, quotients that fp32 holds."""
    x = torch.zeros(64, 64, device="cuda")
    n = np.arange(64)
    token, _ = run(lib, x, n / 64)
    assert (token == n).all()
    token, _ = run(lib, x, np.nextafter(np.float32(n / 64 + 1 / 64), np.float32(0)))
    assert (token == n).all()
    # less than p of the weight before it: with p = n / 64 tokens 0 .. n - 1 are kept
    p = np.maximum(n, 1) / 64
    token, logprob = run(lib, x, np.full(64, 1 - 2.0 ** -24), top_p=p)
    assert (token == np.maximum(n, 1) - 1).all()
    assert np.allclose(logprob, -np.log(np.maximum(n, 1)), rtol=2.0 ** -21, atol=0)
    # p a little more: one more token
    token, _ = run(lib, x, np.full(64, 1 - 2.0 ** -24), top_p=np.nextafter(np.float32(p), np.float32(1)))
    assert (token == np.maximum(n, 1)).all()


def test_masked_rows_and_values(lib):
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((9, 3001)).astype(np.float32)).cuda()
    inf = float("inf")
    x[0] = -inf
    x[1] = float("nan")
    x[2, ::2] = -inf
    x[3, 1::2] = float("nan")
    x[4] = -inf
    x[4, 2777] = -3e38
    x[5, 100], x[5, 2000] = inf, inf
    x[6, :] = -inf
    x[6, [3, 2999]] = 4.0
    x[7] = -0.0
    x[7, ::3] = 0.0
    x[8, 17] = 3.4e38
    x[8, 18] = -3.4e38
    for kw in (dict(), dict(top_k=[5] * 9), dict(top_p=[0.6] * 9), dict(top_k=[1] * 9), dict(temperature=[0.0] * 9),
               dict(top_k=[4] * 9, top_p=[0.9] * 9, min_p=[0.2] * 9), dict(min_p=[1.0] * 9)):
        for u in (0.0, 0.4, 0.999):
            check(lib, x, [u] * 9, **kw)


def test_parameters_at_their_ends(lib):
    rng = np.random.default_rng(7)
    nan, inf = float("nan"), float("inf")
    V = 777
    for name, values in dict(temperature=[0.0, -1.0, nan, 1e-40, 2.0 ** -60, 1e-3, 1e3, 2.0 ** 60, inf],
                             top_k=[0, -1, -2 ** 31, 1, 2, V - 1, V, V + 1, 2 ** 31 - 1],
                             top_p=[0.0, -0.5, nan, 1.0, 7.0, 1e-30, 1e-45, 1 - 2.0 ** -24, inf],
                             min_p=[0.0, -0.5, nan, 1.0, 7.0, 1e-30, 0.999, 2.0 ** -43, inf]).items():
        x = torch.from_numpy(rng.standard_normal((9, V)).astype(np.float32)).cuda()
        check(lib, x, rng.random(9), **{name: values})
        check(lib, x, rng.random(9), **dict({"top_k": [20] * 9, "top_p": [0.8] * 9}, **{name: values}))
    x = torch.from_numpy(rng.standard_normal((6, V)).astype(np.float32)).cuda()
    for kw in (dict(), dict(top_k=[9] * 6)):
        check(lib, x, [0.0, -1.0, nan, 1.0, 5.0, 1e-45], **kw)


def test_logits_of_every_offset(lib):
    """Weights depend on differences alone: large offsets lose nothing that the logits hold."""
    rng = np.random.default_rng(8)
    for off in (0.0, 1000.0, -1e5, 3e7):
        x = torch.from_numpy((off + np.round(rng.standard_normal((20, 5000)) * 3, 1)).astype(np.float32)).cuda()
        check(lib, x, rng.random(20), temperature=rng.uniform(0.3, 2, 20), top_p=[0.9] * 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_any_stride(lib, dtype):
    rng = np.random.default_rng(9)
    base = torch.from_numpy(rng.standard_normal((7, 20011)).astype(np.float32)).cuda().to(dtype)
    for a, b in ((1, 20002), (3, 10), (0, 20011), (4, 20004)):
        check(lib, base[:, a:b], rng.random(7), **_mixed(rng, 7))


@pytest.mark.parametrize("rows", [0, 1, 5, 12, 40])
def test_rows_behind_the_last_are_left(lib, rows):
    rng = np.random.default_rng(10)
    x = torch.from_numpy(rng.standard_normal((12, 999)).astype(np.float32)).cuda()
    u = rng.random(12)
    every, lp = run(lib, x, u, top_p=[0.9] * 12)
    token, logprob = run(lib, x, u, top_p=[0.9] * 12, rows=torch.tensor([rows], dtype=torch.int32, device="cuda"))
    assert (token[:rows] == every[:rows]).all() and (logprob[:rows] == lp[:rows]).all()
    assert (token[rows:] == -7).all() and (logprob[rows:] == 7).all()


def test_frequencies(lib):
    """4,096 numbers spread evenly over a row's distribution hit every token as often as its probability says, to one."""
    rng = np.random.default_rng(11)
    row = (rng.standard_normal(1500) * 2).astype(np.float32)
    n = 4096
    x = torch.from_numpy(row).cuda().expand(n, 1500).contiguous()
    token, logprob = run(lib, x, (np.arange(n) + 0.5) / n, temperature=np.full(n, 0.7))
    p = np.exp((row - row.max()).astype(np.float64) / np.float32(0.7))
    p /= p.sum()
    assert (np.abs(np.bincount(token, minlength=1500) - n * p) <= 1.0).all()
    assert np.allclose(logprob, np.log(p[token]), rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3, 1000, 9001, 32000, 64000])
def test_rows_do_not_depend_on_their_batch(lib, dtype, V):
    """A row of a large batch, where it has fewer CTAs, gives what it gives alone, to the bit."""
    rng = np.random.default_rng(V)
    R = 700
    x = torch.from_numpy((rng.standard_normal((R, V)) * rng.uniform(0.5, 6, (R, 1))).astype(np.float32)).cuda().to(dtype)
    u, kw = rng.random(R), _mixed(rng, R)
    for names in ((), ("temperature", "top_k"), ("temperature", "top_p"), tuple(kw)):
        args = {n: kw[n] for n in names}
        token, logprob = run(lib, x, u, **args)
        for a in range(0, R, 100):
            t, lp = run(lib, x[a:a + 3], u[a:a + 3], **{n: v[a:a + 3] for n, v in args.items()})
            assert (t == token[a:a + 3]).all() and (lp == logprob[a:a + 3]).all()
        check(lib, x[:60], u[:60], **{n: v[:60] for n, v in args.items()})
    parts = [run(lib, x[a:a + 14], u[a:a + 14], top_p=kw["top_p"][a:a + 14]) for a in range(0, R, 14)]
    token, logprob = run(lib, x, u, top_p=kw["top_p"])
    assert (np.concatenate([t for t, _ in parts]) == token).all() and (np.concatenate([lp for _, lp in parts]) == logprob).all()


@pytest.mark.parametrize("V,sigma", [(20000, 1.5), (150000, 3.0), (1500, 4.0)])
def test_borders_at_the_edges_of_bins(lib, V, sigma):
    """p Z within an fp32 rounding of p of the mass above a 1/32 octave's edge, where the leading bits of
    the weights may point at the bin's neighbour."""
    rng = np.random.default_rng(V)
    row = (rng.standard_normal(V) * sigma).astype(np.float32)
    x = np.sort(row.astype(np.float64))[::-1]
    w = np.exp(x - x[0])
    below = np.ceil(x[0] * np.log2(np.e)) * 64 - np.rint(64 * x * np.log2(np.e))
    cum = np.cumsum(w) / w.sum()
    edges = np.flatnonzero(np.diff((below.astype(int) + 63) >> 1))
    edges = edges[(cum[edges] > 0.01) & (cum[edges] < 0.995)]
    p = cum[edges][rng.permutation(edges.size)[:120]].astype(np.float32)
    p = np.concatenate([p, np.nextafter(p, np.float32(0)), np.nextafter(p, np.float32(1))])
    many = torch.from_numpy(row).cuda().expand(p.size, V).contiguous()
    check(lib, many, rng.random(p.size), top_p=p)
    few = slice(0, p.size, 7)
    check(lib, many[few].contiguous(), rng.random(p[few].size), top_p=p[few], min_p=np.full(p[few].size, 1e-3))


def test_streams_graphs_and_equal_calls(lib):
    rng = np.random.default_rng(12)
    R, V = 30, 30001
    x = torch.from_numpy(rng.standard_normal((R, V)).astype(np.float32) * 3).cuda()
    u = torch.from_numpy(rng.random(R).astype(np.float32)).cuda()
    p = torch.full((R,), 0.95, device="cuda")
    token, logprob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    plan = lib.make_sample(x, u, token, logprob=logprob, top_p=p)
    lib.idx_sample(plan)
    want, lp = token.clone(), logprob.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    token.zero_()
    torch.cuda.synchronize()
    lib.idx_sample(plan, stream=side)
    side.synchronize()
    assert torch.equal(token, want) and torch.equal(logprob, lp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.idx_sample(plan)
    x.mul_(0.5)
    u.copy_(torch.rand(R, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    replayed = token.clone()
    lib.idx_sample(plan)
    assert torch.equal(token, replayed)
    # two calls at once, on two streams
    other = torch.empty_like(token)
    plan2 = lib.make_sample(x, u, other, top_p=p)
    torch.cuda.synchronize()
    for _ in range(20):
        lib.idx_sample(plan, stream=side)
        lib.idx_sample(plan2)
    torch.cuda.synchronize()
    assert torch.equal(token, replayed) and torch.equal(other, replayed)
