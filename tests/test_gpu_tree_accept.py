"""idx_tree_accept and idx_tree_commit against plain walks and moves, bit for bit."""
import numpy as np
import pytest
import torch

from tests.tree_util import random_tree

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def walk(parent, draft, target):
    """Accepted token numbers of one request."""
    if not len(draft):
        return []
    got = [0]
    while True:
        c = [u for u in range(1, min(len(draft), 64)) if parent[u] == got[-1] and draft[u] == target[got[-1]]]
        if not c:
            return got
        got.append(c[0])


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Trees:
    """Requests of `new` drafted tokens behind `ctx` cached ones; vocabularies of `words` tokens, so that walks go on."""

    def __init__(self, lib, ctx, new, words=2, chain=False, seed=0, cap=None, stride=None, free=5, free_cap=None):
        self.lib, rng = lib, np.random.default_rng(seed)
        self.ctx, self.new, Q, R = list(ctx), list(new), len(ctx), sum(new)
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.cap = cap or max(R, 1)
        self.parent = [random_tree(rng, n) if not chain else [t - 1 for t in range(n)] for n in new]
        self.draft = [rng.integers(0, words, n) for n in new]
        self.target = [rng.integers(0, words, n) for n in new]
        self.pages = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new)]
        self.P = sum(self.pages) + free + 3
        perm = rng.permutation(self.P)
        self.table = np.full((Q, stride or max(self.pages + [1]) + 1), -1)
        at = 0
        for i, n in enumerate(self.pages):
            self.table[i, :n] = perm[at:at + n][:self.table.shape[1]]
            at += n
        self.free = np.full(free_cap if free_cap is not None else self.P, -5)
        self.free[:free] = perm[at:at + free]
        self.count = free
        flat = lambda x, fill: np.concatenate([np.concatenate(x) if R else [], np.full(self.cap - R, fill)])  # noqa: E731
        self.d = dict(row_start=i32(self.start), draft=i32(flat(self.draft, 0)), target=i32(flat(self.target, 0)), ctx_len=i32(ctx),
                      page_table=i32(self.table), free_pages=i32(self.free), free_count=i32([free]))
        self.d["parent"] = None if chain else i32(flat(self.parent, -1))
        self.o = {n: i32(np.full(k, -9)) for n, k in (("new_ctx", Q), ("accept_len", Q), ("last", Q), ("path", self.cap), ("token", self.cap), ("free_left", 1))}
        self.state = lib.alloc_state(lib.tree_accept_state_size())

    def run(self, stream=None, **kw):
        plan = self.lib.make_tree_accept(**dict(self.d, **self.o, P=self.P, **kw))
        self.lib.idx_tree_accept(plan, self.state, stream)
        return plan

    def check(self):
        o = {n: t.cpu().numpy() for n, t in self.o.items()}
        free, pushed = self.free.copy(), self.count
        for i, n in enumerate(self.new):
            a = self.start[i]
            got = walk(self.parent[i], self.draft[i], self.target[i])
            assert o["accept_len"][i] == len(got) and o["new_ctx"][i] == self.ctx[i] + len(got)
            assert o["path"][a:a + n].tolist() == got + [-1] * (n - len(got))
            assert o["token"][a:a + n].tolist() == [self.target[i][u] for u in got] + [-1] * (n - len(got))
            assert o["last"][i] == (self.target[i][got[-1]] if got else -1)
            for j in range((self.ctx[i] + len(got) + PAGE - 1) // PAGE, min(self.pages[i], self.table.shape[1])):
                if self.table[i, j] >= 0 and pushed < len(free):
                    free[pushed] = self.table[i, j]
                    pushed += 1
        assert (o["path"][self.start[-1]:] == -9).all() and (o["token"][self.start[-1]:] == -9).all()
        assert o["free_left"][0] == pushed and (self.d["free_pages"].cpu().numpy() == free).all()
        assert (self.d["page_table"].cpu().numpy() == self.table).all()


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("words", [1, 2, 5])
@pytest.mark.parametrize("Q", [1, 3, 9, 200, 4096])
def test_paths_and_pages(lib, chain, words, Q):
    rng = np.random.default_rng(Q + words)
    new = rng.integers(0 if Q > 1 else 1, 65, Q)
    ctx = rng.integers(0, 300, Q)
    t = Trees(lib, ctx, new, words, chain, seed=Q, cap=int(new.sum()) + 5)
    t.run()
    t.check()
    assert lib.last_device_status(t.state) == lib.IDX_OK
    for o in t.o.values():      # the state is used again
        o.fill_(-9)
    t.d["free_pages"].copy_(i32(t.free))
    t.run()
    t.check()


def test_ends_of_pages_and_trees(lib):
    """Lengths around pages; full trees and paths through tokens 31 to 33 and 63."""
    for ctx in ([0, 63, 64, 65, 127, 128, 1], [62, 61, 1, 0, 192, 60, 64]):
        for words in (1, 3):
            t = Trees(lib, ctx, [64, 1, 2, 63, 33, 32, 0], words, True, seed=3)
            t.run()
            t.check()
            t = Trees(lib, ctx, [64, 1, 2, 63, 33, 32, 0], words, False, seed=4)
            t.run()
            t.check()


def test_the_first_of_equal_children(lib):
    t = Trees(lib, [10], [8], seed=5)
    t.parent = [[-1, 0, 0, 0, 2, 2, 1, 3]]
    t.draft = [[9, 4, 7, 7, 5, 5, 1, 1]]
    t.target = [[7, 0, 5, 1, 3, 8, 2, 2]]
    for n in ("parent", "draft", "target"):
        t.d[n] = i32(getattr(t, n)[0])
    t.run()
    t.check()
    assert t.o["path"][:4].tolist() == [0, 2, 4, -1] and t.o["last"].item() == 3


def test_in_place(lib):
    t = Trees(lib, [100, 30, 64], [40, 64, 3], 2, seed=6)
    t.o["new_ctx"], t.o["free_left"] = t.d["ctx_len"], t.d["free_count"]
    t.run()
    t.check()


def test_what_is_found_on_the_device(lib):
    def status(t):
        t.run()
        return lib.last_device_status(t.state)

    t = Trees(lib, [10, 20], [8, 8], 1, seed=7)             # a parent that comes later: nobody's child
    t.parent[0][3], t.parent[1][5] = 3, -2
    t.d["parent"] = i32(np.concatenate(t.parent))
    t.parent[0][3] = t.parent[1][5] = -1
    assert status(t) == lib.IDX_EDEVICE
    t.check()
    t = Trees(lib, [10, 20, 5], [8, 70, 3], 1, True, seed=8)   # more than 64 rows
    assert status(t) == lib.IDX_EDEVICE
    t.check()
    t = Trees(lib, [60, 60], [64, 64], 50, True, seed=9)       # a page without an id
    t.table[0, 1] = -1
    t.d["page_table"] = i32(t.table)
    assert status(t) == lib.IDX_EDEVICE
    t.check()
    t = Trees(lib, [60, 60], [64, 64], 50, True, seed=10, free=5, free_cap=6)   # no room on the stack
    assert status(t) == lib.IDX_EDEVICE
    t.check()
    t = Trees(lib, [60, 60], [64, 64], 50, True, seed=11, stride=1)   # a table shorter than its requests
    t.run()
    t.check()
    # rows outside the arrays are cut
    t = Trees(lib, [10, 20, 30], [4, 4, 4], 1, True, seed=12)
    for starts in ([0, 4, 8, 14], [-3, 4, 8, 12], [0, 8, 4, 12], [0, -2 ** 31, 2 ** 31 - 1, 12]):
        t.d["row_start"] = i32(starts)
        t.d["free_pages"].copy_(i32(t.free))
        assert status(t) == lib.IDX_EDEVICE
        assert int(t.o["accept_len"].max()) <= 12 and int(t.o["accept_len"].min()) >= 0


def test_accept_on_streams_and_in_graphs(lib):
    t = Trees(lib, [100, 30, 64, 7], [40, 64, 3, 20], 2, seed=13)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t.run(side)
    side.synchronize()
    t.check()
    plan = t.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.idx_tree_accept(plan, t.state)
    for o in t.o.values():
        o.fill_(-9)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    t.check()


class Cache:
    def __init__(self, lib, P, Hkv, D, kv, layout, keys_alone=False, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shape = (P, Hkv, PAGE, D) if layout == "head" else (P, PAGE, Hkv, D)
        e = torch.bfloat16 if kv == "bf16" else torch.uint8
        both = [torch.randint(0, 256, shape, device="cuda", generator=gen).to(e) for _ in "kv"]
        self.k, self.v = [x.transpose(1, 2) if layout == "head" else x for x in both]
        self.ks, self.vs = [torch.rand(P, Hkv, PAGE, device="cuda", generator=gen) if kv == "e4m3" else None for _ in "kv"]
        if keys_alone:
            self.v = self.vs = None
        self.cache = lib.make_kv_cache(self.k, self.v, self.ks, self.vs)

    def tensors(self):
        return [x for x in (self.k, self.v, self.ks, self.vs)]

    def moved(self, pairs):
        """Copies of the tensors with every (from, to) slot moved at once."""
        a, b = (torch.tensor([p[n] for p in pairs], device="cuda", dtype=torch.long) for n in (0, 1))
        got = []
        for x in (self.k, self.v):
            y = None if x is None else x.clone()
            if y is not None and len(pairs):
                y[b // PAGE, b % PAGE] = x[a // PAGE, a % PAGE]
            got.append(y)
        for x in (self.ks, self.vs):
            y = None if x is None else x.clone()
            if y is not None and len(pairs):
                y[b // PAGE, :, b % PAGE] = x[a // PAGE, :, a % PAGE]
            got.append(y)
        return got


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_moves(lib, kv, D, layout, Hkv):
    rng = np.random.default_rng(D + Hkv)
    new = [1, 64, 0, 13, 40, 64, 7]
    start = np.concatenate([[0], np.cumsum(new)])
    R = sum(new)
    c = Cache(lib, 7, Hkv, D, kv, layout, seed=Hkv)
    slot = rng.permutation(7 * PAGE)[:R]
    path, length = np.full(R, -1), []
    for i, n in enumerate(new):
        if i == 5:
            got = list(range(64))                # everything accepted: nothing moves
        elif i == 1:
            got = [0] + list(range(2, 64))       # all but one: everything moves by one
        else:
            got = [0] + sorted(rng.permutation(n - 1)[:rng.integers(0, n)] + 1) if n else []
        length.append(len(got))
        path[start[i]:start[i] + len(got)] = got
    pairs = [(slot[start[i] + path[start[i] + a]], slot[start[i] + a]) for i in range(len(new)) for a in range(length[i])
             if path[start[i] + a] > a]
    want = c.moved(pairs)
    lib.idx_tree_commit(c.cache, i32(start), i32(length), i32(path), i32(slot))
    for x, y in zip(c.tensors(), want):
        assert (x is None and y is None) or torch.equal(x, y)


def test_moves_that_have_no_place(lib):
    c = Cache(lib, 4, 2, 128, "bf16", "token")
    before = c.moved([])
    start, length = i32([0, 4, 8]), i32([4, 4])
    n = 4 * PAGE
    for path, slot in (([0, 1, 2, 3] * 2, range(8)), ([0, 0, 1, 2] * 2, range(8)), ([0, 4, 70, 2 ** 31 - 1] * 2, range(8)),
                       ([0, -1, -2 ** 31, -5] * 2, range(8)), ([0, 2, 3, -1] * 2, [-1, n, 2 ** 31 - 1, -2 ** 31] * 2)):
        lib.idx_tree_commit(c.cache, start, length, i32(path), i32(list(slot)))
    lib.idx_tree_commit(c.cache, start, i32([-5, 0]), i32([0, 2, 3, -1] * 2), i32(range(8)))
    for starts in ([4, 0, -7], [9, 10, 12], [-5, -4, -3]):      # no rows of the arrays
        lib.idx_tree_commit(c.cache, i32(starts), length, i32([0, 2, 3, -1] * 2), i32(range(8)))
    for x, y in zip(c.tensors(), before):
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_keys_alone(lib, kv):
    c = Cache(lib, 3, 1, 128, kv, "token", True, seed=3)
    # row 2's slot, 7, is read for row 1 before row 4 moves there
    want = c.moved([(7, 5), (9, 7)])
    lib.idx_tree_commit(c.cache, i32([0, 5]), i32([3]), i32([0, 2, 4, -1, -1]), i32([3, 5, 7, 6, 9]))
    for x, y in zip(c.tensors(), want):
        assert (x is None and y is None) or torch.equal(x, y)
