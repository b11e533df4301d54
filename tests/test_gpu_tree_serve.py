"""The calls of a serving loop together: tables, norm and rotation into both caches, ranking,
attention, sampling, acceptance and commit, step by step, eager and as a replayed graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests.test_gpu_sample import reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    spec = importlib.util.spec_from_file_location("tree_serve", os.path.join(ROOT, "examples", "tree_serve.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def walk(tree, draft, target):
    path = [0]
    while True:
        n = next((c for c in range(len(tree)) if tree[c] == path[-1] and draft[c] == target[path[-1]]), None)
        if n is None:
            return path
        path.append(n)


@pytest.mark.parametrize("prompts", [(3000, 1100, 64, 1), (1, 2, 65, 66, 129, 500, 120, 4000, 63)])
def test_a_serving_loop(example, prompts):
    steps, lengths = 14, []

    def each(s):
        ctx, count = s.ctx.cpu().numpy(), s.accept_len.cpu().numpy()
        draft, target, path, token = (x.view(s.Q, s.T).cpu().numpy() for x in (s.draft, s.target, s.path, s.token))
        x, u = s.logits.double().cpu().numpy(), s.u.double().cpu().numpy()
        par = [p.double().cpu().numpy() for p in (s.temperature, s.top_p, s.min_p)]
        k = s.top_k.cpu().numpy()
        for r in range(s.R):       # (logits at temperatures and u of fp32: as in the sampler's own tests)
            want, lp = reference(x[r], par[0][r], int(k[r]), par[1][r], par[2][r], u[r])
            assert target[r // s.T, r % s.T] == want
            assert abs(float(s.logprob[r]) - lp) <= 2.0 ** -21 * abs(lp) + x.shape[1] * 2.0 ** -43
        held = []
        for i in range(s.Q):
            want = walk(example.TREE, draft[i], target[i])
            assert count[i] == len(want) and path[i].tolist() == want + [-1] * (s.T - len(want))
            assert token[i].tolist() == [target[i][n] for n in want] + [-1] * (s.T - len(want))
            assert int(s.last[i]) == target[i][want[-1]] == int(s.token0[i])
            held += s.page_table[i, :-(-ctx[i] // 64)].tolist()
        free = s.free_pages[:int(s.free_count)].tolist()
        assert sorted(held + free) == list(range(s.P))     # no page lost, none held twice
        lengths.append(count.copy())

    s, text = example.main(prompts=prompts, steps=steps, graph=False, each=each, verbose=False)
    total = np.sum(lengths, 0)
    assert (s.ctx.cpu().numpy() == np.array(prompts) - 1 + total).all() and total.max() > steps + 5
    assert [len(t) for t in text] == [n + 1 for n in s.ctx.tolist()]

    # the caches hold what writing the confirmed tokens at their positions gives, to the bit
    lib = example.lib
    pos = torch.cat([torch.arange(n) for n in s.ctx.tolist()]).int().cuda()
    tokens = torch.tensor(sum((t[:-1] for t in text), [])).cuda()
    req = torch.repeat_interleave(torch.arange(s.Q, device="cuda"), s.ctx.long())
    slot = s.page_table[req, pos.long() // 64] * 64 + pos % 64
    mine = [s.k, s.v, s.k_scale, s.v_scale, s.idx_k, s.idx_scale]
    fresh = [torch.zeros_like(t) for t in mine]
    s.prepare(tokens, pos, slot, lib.make_kv_cache(*fresh[:4]), lib.make_kv_cache(fresh[4], None, fresh[5], None))
    page, at = slot.long() // 64, slot.long() % 64
    for a, b in zip(mine, fresh):
        pick = (lambda t: t[page, at]) if a.dtype == torch.uint8 else (lambda t: t[page, :, at])
        assert torch.equal(pick(a), pick(b))

    # the same as replays of one graph
    again, same = example.main(prompts=prompts, steps=steps, graph=True, verbose=False)
    assert same == text and torch.equal(again.ctx, s.ctx) and torch.equal(again.free_pages[:int(again.free_count)], s.free_pages[:int(s.free_count)])
    for t, want in zip((again.k, again.v, again.k_scale, again.v_scale, again.idx_k, again.idx_scale), mine):
        pick = (lambda t: t[page, at]) if t.dtype == torch.uint8 else (lambda t: t[page, :, at])
        assert torch.equal(pick(t), pick(want))


CAPTURED_FIRST = """
import torch, sparse_attention_indexer_launch_gb300 as lib
torch.manual_seed(0)
i32 = dict(dtype=torch.int32, device="cuda")
x = torch.randn(5, 6, 128, device="cuda").bfloat16()
q, cache = torch.zeros(5, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 64, 1, 128, dtype=torch.bfloat16, device="cuda")
values = cache.clone()
norm = lib.make_norm_rope(x[:, :4], x[:, 4:5], x[:, 5:], q_out=q, pos=torch.arange(5, **i32), inv_freq=torch.rand(64, device="cuda"),
                          cache=lib.make_kv_cache(cache, values), slot=torch.arange(5, **i32))
logits, token = torch.randn(5, 5000, device="cuda"), torch.zeros(5, **i32)
sample = lib.make_sample(logits, torch.rand(5, device="cuda"), token, top_p=torch.full((5,), 0.9, device="cuda"))
row_start, table, stack = torch.tensor([0, 5], **i32), torch.tensor([[0, 1]], **i32), torch.zeros(2, **i32)
n = {k: torch.zeros(s, **i32) for k, s in dict(new_ctx=1, accept_len=1, last=1, path=5, token=5, free_left=1).items()}
state = lib.alloc_state(lib.tree_accept_state_size())
accept = lib.make_tree_accept(row_start, token.clone(), token, torch.zeros(1, **i32), table, stack, torch.zeros(1, **i32), P=2, **n)
def calls():
    lib.idx_norm_rope(norm)
    lib.idx_sample(sample)
    lib.idx_tree_accept(accept, state)
    lib.idx_tree_commit(norm.cache, row_start, n["accept_len"], n["path"], slots)
slots = torch.arange(5, **i32)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (q, cache, token, *n.values())]
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (q, cache, token, *n.values())))
print("the same")
"""


def test_first_calls_inside_a_capture():
    """A process whose very first calls are captured: what they set up once works there as well."""
    import subprocess
    import sys
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    done = subprocess.run([sys.executable, "-c", CAPTURED_FIRST], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and "the same" in done.stdout, done.stderr[-2000:]
