"""The calls at the verify step's ends between streams: they start early beside the kernel before them in
their stream, and still wait for what another stream's event says."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


class Step:
    """Every call on small inputs, and a producer on another stream that takes its time."""

    def __init__(self, lib, seed):
        self.lib, g = lib, torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.x = torch.zeros(6, 6, 128, dtype=torch.bfloat16, device="cuda")
        self.logits, self.u = torch.zeros(6, 5000, device="cuda"), torch.zeros(6, device="cuda")
        self.new_x, self.new_logits = torch.randn(6, 6, 128, device="cuda", generator=g).bfloat16(), torch.randn(6, 5000, device="cuda", generator=g)
        self.new_u = torch.rand(6, device="cuda", generator=g)
        self.work = torch.randn(2048, 2048, device="cuda", generator=g)
        self.q = torch.zeros(6, 4, 128, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.zeros(2, 64, 1, 128, dtype=torch.uint8, device="cuda") for _ in "kv")
        ks, vs = (torch.zeros(2, 1, 64, device="cuda") for _ in "kv")
        self.slot, self.starts = torch.arange(6, **i32), torch.tensor([0, 6], **i32)
        self.cache = lib.make_kv_cache(k, v, ks, vs)
        self.norm = lib.make_norm_rope(self.x[:, :4], self.x[:, 4:5], self.x[:, 5:], q_out=self.q, pos=torch.arange(6, **i32),
                                       inv_freq=torch.rand(64, device="cuda", generator=g), cache=self.cache, slot=self.slot)
        self.token, self.draft, self.parent = torch.zeros(6, **i32), torch.zeros(6, **i32), torch.tensor([-1, 0, 0, 2, 2, 4], **i32)
        self.on_path = torch.tensor([True, False, True, False, True, True], device="cuda")
        self.sample = lib.make_sample(self.logits, self.u, self.token, top_p=torch.full((6,), 0.9, device="cuda"))
        self.o = {n: torch.zeros(s, **i32) for n, s in dict(new_ctx=1, accept_len=1, last=1, path=6, token=6, free_left=1).items()}
        self.accept = lib.make_tree_accept(self.starts, self.draft, self.token, torch.zeros(1, **i32), torch.tensor([[0, 1]], **i32),
                                           torch.zeros(2, **i32), torch.zeros(1, **i32), P=2, parent=self.parent, **self.o)
        self.state = lib.alloc_state(lib.tree_accept_state_size())
        self.outs = [self.q, k, v, ks, vs, self.token, *self.o.values()]

    def reset(self):
        for t in (self.x, self.logits, self.u, self.draft, *self.outs):
            t.zero_()

    def produce(self):
        y = self.work
        for _ in range(24):
            y = torch.mm(y, self.work) * 0.02
        self.x.copy_(self.new_x)
        self.logits.copy_(self.new_logits)
        self.u.copy_(self.new_u)

    def calls(self):
        lib = self.lib
        lib.idx_norm_rope(self.norm)
        lib.idx_sample(self.sample)
        self.draft.copy_(torch.where(self.on_path, self.token[self.parent.clamp(min=0).long()], -1))
        lib.idx_tree_accept(self.accept, self.state)
        lib.idx_tree_commit(self.cache, self.starts, self.o["accept_len"], self.o["path"], self.slot)

    def crossed(self):
        """A first round of calls, then, behind another stream's producer, a second: no kernel in between."""
        here, side = torch.cuda.current_stream(), torch.cuda.Stream()
        side.wait_stream(here)
        self.calls()                     # on zeros
        with torch.cuda.stream(side):
            done = torch.cuda.Event()
            side.wait_stream(here)
            self.produce()
            done.record(side)
        self.lib.idx_tree_commit(self.cache, self.starts, self.o["accept_len"], self.o["path"], self.slot)
        here.wait_event(done)
        self.calls()


def test_events_of_other_streams(lib):
    s = Step(lib, 1)
    s.reset()
    s.produce()
    s.calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in s.outs]
    assert s.o["path"].tolist() == [0, 2, 4, 5, -1, -1] and bool(s.q.any())
    for _ in range(5):
        s.reset()
        s.crossed()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outs, want))
    s.reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.crossed()
    for _ in range(5):
        s.reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outs, want))
