"""idx_norm_rope against the formulas of include/idx.h in 64 bits.

Tolerances: an output is rounded once (half a step: bf16 2^-8, E4M3 2^-4 of the value, and
2^-10 of the scale among E4M3's subnormals).  Before that a value z = inv (x A + x' B) + C
sees at most 16 fp32 roundings (2^-24 each: products of weights and angles, the sum of
squares, its root, the sums), an angle off by pi 2^-24 and, for LayerNorm, a mean off by
2^-22 of the largest |x|: together less than 2^-19 (|y| + |y'| + inv max |x|)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


class Case:
    """Inputs of a call: fused rows [R][Hq + 2 Hkv][D] with `pad` elements behind each row."""

    def __init__(self, lib, R=5, Hq=5, Hkv=3, D=128, kv="bf16", norm=1, k_norm=1, rot=None, interleaved=False, axes=1,
                 seed=0, pad=0, layout="token", weights=True, amp=1.0):
        self.lib, self.R, self.Hq, self.Hkv, self.D, self.kv = lib, R, Hq, Hkv, D, kv
        self.norm, self.k_norm, self.rot, self.il, self.eps = norm, k_norm, D if rot is None else rot, interleaved, 1e-5
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        H = Hq + 2 * Hkv
        flat = torch.randn(R, H * D + pad, device="cuda", generator=gen).mul_(amp).add_(0.25 * amp).bfloat16()
        x = flat[:, :H * D].unflatten(1, (H, D))
        self.x = x
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        w = lambda on: torch.randn(D, device="cuda", generator=gen) if on and weights else None  # noqa: E731
        self.qw, self.kw = w(norm != 0), w(k_norm != 0)
        self.qb, self.kb = w(norm == 2), w(k_norm == 2)
        self.inv = torch.from_numpy((1e4 ** (-np.arange(self.rot // 2) * 2.0 / max(self.rot, 1))).astype(np.float32)).cuda()
        self.axis = rng.integers(0, axes, self.rot // 2).tolist()
        pos = rng.integers(0, 1 << 20, (axes, R))
        pos[0, :min(R, 4)] = [0, 2 ** 31 - 1, -7, 524287][:min(R, 4)]
        self.pos = torch.from_numpy(pos.astype(np.int32)).cuda()
        self.q_out = torch.full((R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if Hq else None
        self.k_out = torch.full((R, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") if Hkv and kv == "none" else None
        self.cache = self.slot = None
        if kv != "none":
            P = (R + PAGE - 1) // PAGE + 2
            self.slot = torch.from_numpy(rng.permutation(P * PAGE)[:R].astype(np.int32)).cuda()
            e = torch.bfloat16 if kv.startswith("bf16") else torch.uint8
            shape = (P, Hkv, PAGE, D) if layout == "head" else (P, PAGE, Hkv, D)
            both = [torch.randint(0, 100, shape, device="cuda", generator=gen).to(e) for _ in "kv"]
            self.K, self.V = [y.transpose(1, 2) if layout == "head" else y for y in both]
            self.ks, self.vs = [torch.rand(P, Hkv, PAGE, device="cuda", generator=gen) if e == torch.uint8 else None for _ in "kv"]
            if kv.endswith("keys"):
                self.V = self.vs = None
            self.cache = lib.make_kv_cache(self.K, self.V, self.ks, self.vs)

    def plan(self, **kw):
        keys = self.V is None if self.kv != "none" else True
        a = dict(q_out=self.q_out, k_out=self.k_out, pos=self.pos, inv_freq=self.inv, axis=self.axis, interleaved=self.il,
                 q_norm=self.norm, k_norm=self.k_norm, q_weight=self.qw, q_bias=self.qb, k_weight=self.kw, k_bias=self.kb,
                 eps=self.eps, cache=self.cache, slot=self.slot)
        a.update(kw)
        return self.lib.make_norm_rope(self.q if self.Hq else None, self.k if self.Hkv else None,
                                       None if keys or not self.Hkv else self.v, **a)

    def exact(self, x, norm, weight, bias):
        """(z, room): the rotated heads in 64 bits, and the fp32 error that the module's text allows."""
        x = x.double().cpu().numpy()
        inv, mean = np.ones(x.shape[:2] + (1,)), np.zeros(x.shape[:2] + (1,))
        if norm == 2:
            mean = x.mean(-1, keepdims=True)
        if norm:
            inv = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + self.eps)
        w = np.ones(self.D) if weight is None else weight.double().cpu().numpy()
        b = np.zeros(self.D) if bias is None else bias.double().cpu().numpy()
        y = (x - mean) * inv * w + b
        room = np.abs(y) + (np.abs(x).max(-1, keepdims=True) * inv * np.abs(w) if norm == 2 else 0) + np.abs(b)
        z, more = y.copy(), room.copy()
        pos, fr = self.pos.cpu().numpy().astype(np.float64), self.inv.cpu().numpy().astype(np.float64)
        for i in range(self.rot // 2):
            a, c = (2 * i, 2 * i + 1) if self.il else (i, i + self.rot // 2)
            t = (pos[self.axis[i]] * fr[i])[:, None]
            z[:, :, a] = y[:, :, a] * np.cos(t) - y[:, :, c] * np.sin(t)
            z[:, :, c] = y[:, :, c] * np.cos(t) + y[:, :, a] * np.sin(t)
            more[:, :, a] = more[:, :, c] = room[:, :, a] + room[:, :, c]
        return z, 2.0 ** -19 * more

    def check(self, rows=None, q_out=None, k_out=None):
        n = self.R if rows is None else rows
        if self.Hq:
            z, room = self.exact(self.q0 if hasattr(self, "q0") else self.q, self.norm, self.qw, self.qb)
            got = (q_out if q_out is not None else self.q_out).double().cpu().numpy()
            assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + room)[:n].all()
        if not self.Hkv:
            return
        z, room = self.exact(self.k0 if hasattr(self, "k0") else self.k, self.k_norm, self.kw, self.kb)
        k_out = k_out if k_out is not None else self.k_out
        if k_out is not None:
            got = k_out.double().cpu().numpy()
            assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + room)[:n].all()
        if self.kv == "none":
            return
        page, off = self.slot.long() // PAGE, self.slot.long() % PAGE
        if self.kv.startswith("bf16"):
            got = self.K[page, off].double().cpu().numpy()
            assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + room)[:n].all()
        else:
            sc = self.ks[page, :, off].double().cpu().numpy()
            amax = np.abs(z).max(-1)
            assert (np.abs(sc - amax / 448) <= 2.0 ** -23 * amax / 448 + room.max(-1) / 448)[:n].all()
            got = self.K.view(torch.float8_e4m3fn)[page, off].double().cpu().numpy() * sc[:, :, None]
            # the code's half step, the scale's error (2^-23 and room / amax of the value) behind it
            tol = 2.0 ** -4 * np.abs(z) + 2.0 ** -10 * sc[:, :, None] + 2 * room + 2.0 ** -22 * np.abs(z)
            assert (np.abs(got - z) <= tol + 2 * room.max(-1, keepdims=True))[:n].all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("norm,k_norm", [(0, 2), (1, 1), (2, 0)])
@pytest.mark.parametrize("part", [0, 1, 2, 3])
def test_formulas(lib, D, il, norm, k_norm, part):
    rot = [0, 16, D // 2, D][part]
    for R, Hq, Hkv in ((1, 1, 1), (9, 5, 3), (67, 0, 2), (3, 33, 0)):
        c = Case(lib, R, Hq, Hkv, D, "none", norm, k_norm, rot, il, axes=1 + part, seed=D + part, pad=8 * part)
        lib.idx_norm_rope(c.plan())
        c.check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "bf16 keys", "e4m3 keys"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_into_the_cache(lib, kv, D, layout):
    for R, Hq, Hkv, rot in ((1, 8, 1, D), (70, 5, 3, D // 2), (131, 0, 16, 0)):
        c = Case(lib, R, Hq, Hkv, D, kv, 1, 2, rot, True, seed=R, layout=layout)
        K0, V0 = c.K.clone(), None if c.V is None else c.V.clone()
        ks0, vs0 = [None if s is None else s.clone() for s in (c.ks, c.vs)]
        lib.idx_norm_rope(c.plan())
        c.check()
        # v as idx_write_kv writes it, and nothing else touched
        page, off = c.slot.long() // PAGE, c.slot.long() % PAGE
        if V0 is not None:
            spare = [x.clone() if x is not None else None for x in (K0, V0, ks0, vs0)]
            lib.idx_write_kv(lib.make_kv_cache(*spare), c.v, c.v, c.slot)
            assert torch.equal(c.V, spare[1]) and (vs0 is None or torch.equal(c.vs, spare[3]))
        K0[page, off] = c.K[page, off]
        assert torch.equal(K0, c.K)
        if ks0 is not None:
            ks0[page, :, off] = c.ks[page, :, off]
            assert torch.equal(ks0, c.ks)


def test_heads_of_a_full_model(lib):
    """Enough rows for warps of many heads, and both ends of the rule that gives a warp its heads."""
    for R in (1, 64, 700):
        c = Case(lib, R, 64, 8, 128, "e4m3", seed=R)
        lib.idx_norm_rope(c.plan())
        c.check()


@pytest.mark.parametrize("kv", ["none", "bf16", "e4m3"])
def test_in_place_and_beside_a_cache(lib, kv):
    c = Case(lib, 40, 6, 2, 128, kv, seed=3, pad=16)
    c.q0, c.k0 = c.q.clone(), c.k.clone()
    v0 = c.v.clone()
    lib.idx_norm_rope(c.plan(q_out=c.q, k_out=c.k))
    c.check(q_out=c.q, k_out=c.k)
    assert torch.equal(c.v, v0)


@pytest.mark.parametrize("rows", [0, 1, 23, 40, 99])
def test_rows_behind_the_last_are_left(lib, rows):
    c = Case(lib, 40, 6, 2, 64, "e4m3", seed=4)
    K0, V0, ks0, vs0 = c.K.clone(), c.V.clone(), c.ks.clone(), c.vs.clone()
    lib.idx_norm_rope(c.plan(rows=torch.tensor([rows], dtype=torch.int32, device="cuda")))
    c.check(rows=rows)
    assert bool((c.q_out[rows:] == 7).all())
    page, off = c.slot.long()[rows:] // PAGE, c.slot.long()[rows:] % PAGE
    for new, old in ((c.K, K0), (c.V, V0)):
        assert torch.equal(new[page, off], old[page, off])
    for new, old in ((c.ks, ks0), (c.vs, vs0)):
        assert torch.equal(new[page, :, off], old[page, :, off])


def test_slots_without_a_place_write_nothing(lib):
    c = Case(lib, 12, 2, 2, 128, "bf16", seed=5)
    K0, V0, n = c.K.clone(), c.V.clone(), c.K.shape[0] * PAGE
    c.slot[:] = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31] * 3, dtype=torch.int32)
    lib.idx_norm_rope(c.plan())
    assert torch.equal(c.K, K0) and torch.equal(c.V, V0)
    z, room = c.exact(c.q, 1, c.qw, None)
    assert (np.abs(c.q_out.double().cpu().numpy() - z) <= 2.0 ** -8 * np.abs(z) + room).all()


@pytest.mark.parametrize("norm", [1, 2])
@pytest.mark.parametrize("amp", [2.0 ** -60, 2.0 ** 70, 2.0 ** 120])
def test_squares_past_the_range(lib, norm, amp):
    c = Case(lib, 6, 4, 2, 128, "none", norm, norm, seed=6, amp=amp)
    lib.idx_norm_rope(c.plan())
    c.check()


def test_infinities_and_nan(lib):
    c = Case(lib, 8, 1, 1, 64, "e4m3", 0, 1, 32, False, seed=7, weights=False)
    c.q[0, 0, 40], c.q[1, 0, 3], c.q[2, 0, 50] = float("inf"), float("nan"), -0.0
    c.k[3, 0, 40], c.k[4, 0, 3] = float("inf"), float("nan")
    c.k[5] = 0
    lib.idx_norm_rope(c.plan())
    page, off = c.slot.long() // PAGE, c.slot.long() % PAGE
    q = c.q_out.float().cpu()
    # without a norm only the pair of the element is touched: 40 and 50 do not turn, 3 turns with 19
    assert q[0, 0, 40] == float("inf") and bool(torch.isfinite(q[0, 0, :40]).all()) and bool(torch.isfinite(q[0, 0, 41:]).all())
    bad = torch.isnan(q[1, 0])
    assert bad[3] and bad[19] and int(bad.sum()) == 2
    assert q[2, 0, 50] == 0 and bool(torch.signbit(q[2, 0, 50]))
    k = c.K.view(torch.float8_e4m3fn)[page, off].float().cpu()
    # an infinite square: inf / inf for the element itself, zeros beside it
    assert torch.isnan(k[3, 0, 40]) and bool((k[3, 0, :40] == 0).all())
    assert bool(torch.isnan(k[4]).all()) and c.ks[page[4], 0, off[4]] == 1
    assert bool((k[5] == 0).all()) and c.ks[page[5], 0, off[5]] == 1
    rest = [6, 7]
    z, room = c.exact(c.k, 1, None, None)
    got = (k[rest].double() * c.ks[page, :, off].double().cpu()[rest][..., None]).numpy()
    sc = c.ks[page, :, off].double().cpu()[rest][..., None].numpy()
    assert (np.abs(got - z[rest]) <= 2.0 ** -4 * np.abs(z[rest]) + 2.0 ** -10 * sc + 4 * room[rest].max()).all()


def test_a_frequency_that_is_not_finite_turns_to_nan(lib):
    c = Case(lib, 2, 1, 0, 64, "none", 0, 0, 32, False, seed=8)
    c.inv[2], c.inv[5] = float("nan"), float("inf")
    lib.idx_norm_rope(c.plan())
    bad = torch.isnan(c.q_out[:, 0])
    assert bool(bad[:, [2, 18, 5, 21]].all()) and int(bad.sum()) == 8


def test_frequencies_of_every_size(lib):
    c = Case(lib, 4, 1, 0, 256, "none", 0, 0, 256, True, seed=9)
    c.inv[:] = torch.from_numpy(np.concatenate([2.0 ** -np.arange(60.0), 2.0 ** -140 * np.ones(4), -(0.7 ** np.arange(64.0))]).astype(np.float32))
    lib.idx_norm_rope(c.plan())
    c.check()


def test_another_stream_and_a_replayed_graph(lib):
    c = Case(lib, 30, 8, 2, 128, "e4m3", seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = c.plan()
    lib.idx_norm_rope(plan, stream=side)
    side.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.idx_norm_rope(plan)
    c.x.copy_(torch.randn(c.x.shape, device="cuda").bfloat16())
    c.pos += 11
    graph.replay()
    torch.cuda.synchronize()
    c.check()


def test_the_indexers_own_cache(lib):
    """Keys alone, as idx_launch reads them: [P][64][128] with a scale per token."""
    c = Case(lib, 50, 64, 1, 128, "e4m3 keys", 0, 2, 64, True, seed=11)
    keys = c.K.view(c.K.shape[0], PAGE, 128)
    lib.idx_norm_rope(c.plan())
    c.check()
    assert keys.data_ptr() == c.cache.k


@pytest.mark.parametrize("Hq,Hkv,norm", [(64, 8, "rms"), (5, 3, "rms"), (64, 1, "layer"), (0, 2, "rms"), (3, 0, "none")])
def test_rows_do_not_depend_on_their_batch(lib, Hq, Hkv, norm):
    """A row's warps and their shares follow from the batch; its values do not, to the bit."""
    gen = torch.Generator(device="cuda").manual_seed(Hq)
    R, D = 9001, 128
    kind = dict(rms=lib.IDX_NORM_RMS, layer=lib.IDX_NORM_LAYER, none=lib.IDX_NORM_NONE)[norm]
    x = torch.randn(R, Hq + Hkv, D, device="cuda", generator=gen).bfloat16()
    pos = torch.randint(-2 ** 31, 2 ** 31, (R,), device="cuda", generator=gen).int()
    inv_freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda").float() / D)
    weight = None if norm == "none" else torch.rand(D, device="cuda", generator=gen)

    def rows(a, b):
        out = torch.full((b - a, Hq + Hkv, D), -7.0, device="cuda").bfloat16()
        part = lambda t, lo, hi: t[:, lo:hi] if hi > lo else None  # noqa: E731
        lib.idx_norm_rope(lib.make_norm_rope(part(x[a:b], 0, Hq), part(x[a:b], Hq, Hq + Hkv), q_out=part(out, 0, Hq), k_out=part(out, Hq, Hq + Hkv),
                                             pos=pos[a:b], inv_freq=inv_freq, q_norm=kind, k_norm=kind, q_weight=weight if Hq else None,
                                             k_weight=weight if Hkv else None))
        return out

    every = rows(0, R)
    for a, b in ((0, 1), (77, 84), (100, 400), (500, 1500), (2000, 5000), (R - 4300, R)):
        assert torch.equal(rows(a, b), every[a:b])
