"""idx_tree_tables and idx_write_kv against plain host computations: whole numbers and
codes equal, nothing else touched, errors found on the device reported."""
import numpy as np
import pytest
import torch

from tests import tree_util as tu

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


class Tables:
    def __init__(self, lib, ctx, new, parents=None, cap=None, stride=None, spare=5, seed=0, with_mask=True, offset=0):
        rng = np.random.default_rng(seed)
        Q, R = len(ctx), sum(max(n, 0) for n in new)
        held = [(max(c, 0) + 63) // 64 for c in ctx]
        full = [(max(c, 0) + max(n, 0) + 63) // 64 for c, n in zip(ctx, new)]
        self.stride = stride if stride is not None else max(full + [1])
        self.cap = R if cap is None else cap
        self.P = sum(full) + max(spare, 0) + 1
        perm = rng.permutation(self.P).astype(np.int32)
        self.table = np.full((Q, self.stride), -1, np.int32)
        at = 0
        for i in range(Q):
            n = min(held[i], self.stride)
            self.table[i, :n] = perm[at:at + n]
            at += held[i]
        need = sum(max(0, min(f, self.stride) - h) for f, h in zip(full, held))
        self.free = perm[at:at + need + spare] if spare >= 0 else perm[at:at + need + spare]
        self.ctx, self.new, self.parents = ctx, new, parents
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        flat = None if parents is None else np.array(sum(parents, []) + [-1] * max(0, self.cap - R), np.int32)[:max(self.cap, 1)]
        mk = lambda n, dt=torch.int32: torch.full((n + offset,), -77, dtype=dt, device="cuda")[offset:]  # noqa: E731
        self.o = dict(row_start=mk(Q + 1), free_left=mk(1), row_req=mk(self.cap), row_bound=mk(self.cap),
                      row_pos=mk(self.cap), slot=mk(self.cap), mask=mk(self.cap, torch.int64) if with_mask else None)
        self.page_table = dev(self.table)
        self.keep = [dev(np.array(ctx, np.int32)), dev(np.array(new, np.int32)), dev(np.append(self.free, 0).astype(np.int32)),
                     dev(np.array([len(self.free)], np.int32)), None if flat is None else dev(flat)]
        self.args = lib.make_tree_tables(self.keep[0], self.keep[1], self.page_table, self.keep[2], self.keep[3],
                                         parent=self.keep[4], P=self.P, **self.o)
        self.state = lib.alloc_state(lib.tree_tables_state_size())

    def expected(self):
        table = self.table.copy()
        free = list(self.free)
        start, rows = [0], []
        for i, (c, n) in enumerate(zip(self.ctx, self.new)):
            c, n = max(c, 0), max(n, 0)
            for k in range((c + 63) // 64, min((c + n + 63) // 64, self.stride)):
                table[i, k] = free.pop() if free else -1
            anc = tu.ancestor_masks(self.parents[i]) if self.parents is not None and n <= 64 else [(2 << t) - 1 if t < 64 else 0 for t in range(n)]
            for t in range(n):
                at = c + t
                page = table[i, at // 64] if at // 64 < self.stride else -1
                depth = bin(anc[t]).count("1") - 1 if t < 64 else t
                rows.append((i, at + 1, c + depth, -1 if page < 0 else page * 64 + at % 64, anc[t]))
            start.append(min(start[-1] + n, self.cap))
        rows = (rows + [(0, 0, 0, -1, 0)] * self.cap)[:self.cap]
        return table, start, len(free), rows

    def check(self):
        table, start, left, rows = self.expected()
        assert np.array_equal(self.page_table.cpu().numpy(), table)
        assert self.o["row_start"].tolist() == start
        assert self.o["free_left"].tolist() == [left]
        for k, name in enumerate(("row_req", "row_bound", "row_pos", "slot")):
            assert self.o[name].tolist() == [r[k] for r in rows], name
        if self.o["mask"] is not None:
            assert self.o["mask"].tolist() == tu.as_int64([r[4] for r in rows])


@pytest.mark.parametrize("offset", [0, 1])
def test_trees_and_chains(lib, offset):
    rng = np.random.default_rng(1)
    ctx = [0, 1, 63, 64, 65, 500, 128, 0, 7, 4096]
    new = [1, 64, 1, 1, 63, 0, 64, 0, 57, 3]
    for parents in (None, [tu.random_tree(rng, n) for n in new]):
        t = Tables(lib, ctx, new, parents, cap=sum(new) + 13, seed=2, offset=offset)
        lib.idx_tree_tables(t.args, t.state)
        assert lib.last_device_status(t.state) == lib.IDX_OK
        t.check()


@pytest.mark.parametrize("Q", [1, 2, 255, 256, 257, 1000, 4096])
def test_request_counts(lib, Q):
    rng = np.random.default_rng(Q)
    ctx = rng.integers(0, 300, Q).tolist()
    new = rng.integers(0, 9, Q).tolist()
    t = Tables(lib, ctx, new, [tu.random_tree(rng, n) for n in new], seed=Q)
    lib.idx_tree_tables(t.args, t.state)
    assert lib.last_device_status(t.state) == lib.IDX_OK
    t.check()


def test_prompts(lib):
    t = Tables(lib, [0, 0, 1000, 0], [70001, 1, 30000, 129], seed=3, with_mask=False)
    lib.idx_tree_tables(t.args, t.state)
    assert lib.last_device_status(t.state) == lib.IDX_OK
    t.check()


def test_all_outputs_hold_on_a_second_call(lib):
    t = Tables(lib, [100, 200], [30, 64], seed=4)
    for _ in range(2):
        lib.idx_tree_tables(t.args, t.state)
        t.check()


@pytest.mark.parametrize("case", ["pages", "table", "cap", "parent", "long", "id", "negative"])
def test_errors_found_on_the_device(lib, case):
    kw = dict(seed=5)
    ctx, new, parents = [100, 60, 10], [40, 60, 3], None
    if case == "pages":
        kw["spare"] = -1
    elif case == "table":
        kw["stride"] = 2
    elif case == "cap":
        kw["cap"] = 70
    elif case == "long":
        new = [40, 70, 3]
    elif case == "parent":
        parents = [[-1] + list(range(n - 1)) for n in new]
    elif case == "negative":
        ctx, new = [-5, 60, 10], [40, -3, 3]
    t = Tables(lib, ctx, new, parents, **kw)
    if case == "parent":       # a parent that is its own token: read as a root
        t.keep[4][40 + 7] = 7
        t.parents[1][7] = -1
    if case == "id":           # a held page outside the cache
        t.page_table[0, 1] = t.P
        t.table[0, 1] = -1
    lib.idx_tree_tables(t.args, t.state)
    st = lib.last_device_status(t.state)
    assert st == (lib.IDX_OK if case == "negative" else lib.IDX_EDEVICE)
    if case == "id":
        t.page_table[0, 1] = -1
    t.check()


def test_tables_refusals(lib):
    t = Tables(lib, [100], [4], seed=6)

    def call(state=None, **kw):
        import ctypes
        a = lib.TreeTables.from_buffer_copy(t.args)
        for k, v in kw.items():
            setattr(a, k, v)
        state = t.state if state is None else state
        return lib.lib.idx_tree_tables(ctypes.byref(a), lib._ptr(state), state.numel(), lib._stream(None))

    for kw in (dict(ctx_len=None), dict(new_len=None), dict(page_table=None), dict(free_pages=None), dict(slot=None),
               dict(Q=0), dict(P=0), dict(pt_stride=0), dict(cap=-1), dict(free_left=t.args.free_count)):
        assert call(**kw) == lib.IDX_EINVAL, kw
    for kw in (dict(Q=4097), dict(P=2 ** 30)):
        assert call(**kw) == lib.IDX_EUNSUPPORTED, kw
    assert call(state=t.state[8:]) == lib.IDX_EINVAL
    assert call(state=t.state[:64]) == lib.IDX_EINVAL
    with pytest.raises(ValueError):
        lib.make_tree_tables(t.keep[0].long(), t.keep[1], t.page_table, t.keep[2], t.keep[3], P=t.P, **t.o)


def _codes(x):
    """E4M3 codes and scales of float32 vectors, by search over the 127 magnitudes."""
    mag = []
    for c in range(127):
        e, m = c >> 3, c & 7
        mag.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    mag = np.array(mag)
    amax = np.abs(x).max(-1)
    sc = np.where(amax > 0, (amax / np.float32(448.0)).astype(np.float32), np.float32(1.0)).astype(np.float32)
    y = (x / sc[..., None]).astype(np.float32).astype(np.float64)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(mag, a), 1, 126)
    lo = hi - 1
    down, up = a - mag[lo], mag[hi] - a
    c = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c | np.where(np.signbit(y), 128, 0)).astype(np.uint8), sc


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,D,R", [(1, 64, 1), (8, 128, 37), (3, 64, 100), (16, 128, 3), (1, 128, 2000)])
@pytest.mark.parametrize("layout", ["token", "head", "pair"])
def test_write(lib, kv, Hkv, D, R, layout):
    rng = np.random.default_rng(R)
    P = R // 64 + 3
    dt = torch.uint8 if kv == "e4m3" else torch.int16
    fill = 0x55 if kv == "e4m3" else 0x5555
    if layout == "head":
        raw = [torch.full((P, Hkv, PAGE, D), fill, dtype=dt, device="cuda") for _ in "kv"]
        k, v = (x.transpose(1, 2) for x in raw)
    elif layout == "pair":
        both = torch.full((P, 2, PAGE, Hkv, D), fill, dtype=dt, device="cuda")
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.full((P, PAGE, Hkv, D), fill, dtype=dt, device="cuda") for _ in "kv")
    ks, vs = (torch.full((P, Hkv, PAGE), 5.0, device="cuda") for _ in "kv") if kv == "e4m3" else (None, None)
    qkv = torch.randn(R, 5 + 2 * Hkv, D, device="cuda").bfloat16()
    new = [qkv[:, 5:5 + Hkv], qkv[:, 5 + Hkv:]]
    new[0][0, 0] = 0.0                                    # an all-zero vector: scale 1
    new[1][-1, 0, :7] = torch.tensor([1e-8, -0.0, 3e38, -3e38, 448.0, 1.0, 0.0], device="cuda").bfloat16()
    slot = rng.permutation(P * PAGE)[:R].astype(np.int32)
    slot[rng.random(R) < 0.1] = -1
    if R > 3:
        slot[1], slot[2] = P * PAGE, 2 ** 31 - 1          # outside the cache: nothing is written
    cache = lib.make_kv_cache(*((x if kv == "e4m3" else x.view(torch.bfloat16)) for x in (k, v)), ks, vs)
    lib.idx_write_kv(cache, new[0], new[1], torch.from_numpy(slot).cuda())
    live = (slot >= 0) & (slot < P * PAGE)
    page, off = slot[live] // 64, slot[live] % 64
    for x, sc, n in ((k, ks, new[0]), (v, vs, new[1])):
        want = np.full((P, PAGE, Hkv, D), fill, np.uint8 if kv == "e4m3" else np.int16)
        if kv == "e4m3":
            c, s = _codes(n.float().cpu().numpy())
            want[page, off] = c[live]
            scales = np.full((P, Hkv, PAGE), 5.0, np.float32)
            scales[page, :, off] = s[live]
            assert np.array_equal(sc.cpu().numpy(), scales)
        else:
            want[page, off] = n.view(torch.int16).cpu().numpy()[live]
        assert np.array_equal(x.cpu().numpy(), want)


def test_write_past_32_bits(lib):
    P = 33000
    k, v = (torch.zeros(P, PAGE, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    new = torch.randn(2, 8, 128, device="cuda").bfloat16()
    slot = torch.tensor([P * PAGE - 1, 5], dtype=torch.int32, device="cuda")
    lib.idx_write_kv(lib.make_kv_cache(k, v), new, new, slot)
    assert torch.equal(k[P - 1, 63], new[0]) and torch.equal(v[0, 5], new[1])
    assert int((k != 0).sum()) == int((new != 0).sum())


def test_write_refusals(lib):
    k, v = (torch.zeros(2, PAGE, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    new = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(3, dtype=torch.int32, device="cuda")
    cache = lib.make_kv_cache(k, v)

    def call(stride=128, R=3, a=new, s=slot, **kw):
        import ctypes
        c = lib.KvCache.from_buffer_copy(cache)
        for n, x in kw.items():
            setattr(c, n, x)
        return lib.lib.idx_write_kv(ctypes.byref(c), lib._ptr(a), lib._ptr(new), stride, lib._ptr(s), R, lib._stream(None))

    assert call() == lib.IDX_OK
    assert call(R=0) == lib.IDX_OK
    for kw in (dict(k=None), dict(P=0), dict(Hkv=0), dict(kv_dtype=9), dict(page_stride=4), dict(token_stride=0),
               dict(k_scale=k.data_ptr()), dict(kv_dtype=lib.IDX_KV_E4M3), dict(R=-1), dict(stride=120), dict(stride=132),
               dict(a=None), dict(s=None), dict(k=k.data_ptr() + 8)):
        assert call(**kw) == lib.IDX_EINVAL, kw
    for kw in (dict(D=96), dict(Hkv=2000, stride=2000 * 64), dict(P=2 ** 30)):
        assert call(**kw) == lib.IDX_EUNSUPPORTED, kw
    with pytest.raises(ValueError):
        lib.idx_write_kv(cache, new.float(), new, slot)
    with pytest.raises(ValueError):
        lib.idx_write_kv(cache, new[:, :1], new, slot)
    with pytest.raises(ValueError):
        lib.idx_write_kv(cache, new, new, slot.long())
