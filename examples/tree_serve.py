"""Verify steps over drafted trees in a loop, every one a replay of one CUDA graph.

A batch of requests with cached prompts drafts a tree of tokens behind its newest one, and a
step confirms as many of them as the model would have drawn itself:
  1. pages, slots, positions and tree masks of the drafted tokens   idx_tree_tables
  2. head norms, rotation and the caches' writes, of the model      idx_norm_rope
     and of the indexer (its keys alone)                            idx_norm_rope
  3. the cached positions that matter to every token                idx_launch
  4. attention to these and to the token's ancestors                idx_tree_attention_selected
  5. a token of every row by its request's temperature, top-k, ...  idx_sample
  6. the path that the drawn tokens confirm, lengths and pages      idx_tree_accept
  7. its keys and values to their places, in both caches            idx_tree_commit
Nothing of a step is known to the host: lengths, pages and tokens stay on the GPU.

The model is one random layer (16 query heads, 2 key/value heads of dimension 128, an E4M3
cache), with the projections of every token's embedding as a table; the draft takes the
tokens that a head on the embedding alone finds likely.  Needs a GB300.

    python examples/tree_serve.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_launch_gb300 as lib  # noqa: E402

HQ, HKV, D, IDX_HEADS, IDX_D, IDX_ROT, K, VOCAB, WIDTH = 16, 2, 128, 64, 128, 64, 2048, 2000, 256
TREE = (-1, 0, 0, 1, 1, 2, 3, 3, 6)         # parents; the children of a token stand in order of likelihood


class Model:
    """Weights, and what they make of every token."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
        embed = normal(VOCAB, WIDTH).bfloat16()
        project = lambda n: (embed.float() @ normal(WIDTH, n) * WIDTH ** -0.5).bfloat16()  # noqa: E731
        self.qkv = project((HQ + 2 * HKV) * D).view(VOCAB, HQ + 2 * HKV, D)
        self.idx_qk = project((IDX_HEADS + 1) * IDX_D).view(VOCAB, IDX_HEADS + 1, IDX_D)
        self.idx_w = torch.rand(VOCAB, IDX_HEADS, device="cuda", generator=g)
        self.q_weight, self.k_weight, self.idx_k_weight = (1 + 0.1 * normal(n) for n in (D, D, IDX_D))
        self.idx_k_bias = 0.1 * normal(IDX_D)
        turns = lambda rot: 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").float() / rot)  # noqa: E731
        self.inv_freq, self.idx_inv_freq = turns(D), turns(IDX_ROT)
        self.out = (normal(HQ * D, VOCAB) * (HQ * D) ** -0.5).bfloat16()
        self.skip = (embed.float() @ normal(WIDTH, VOCAB) * 2 * WIDTH ** -0.5).bfloat16()
        children = max(TREE.count(p) for p in range(len(TREE)))
        self.likely = self.skip.float().topk(children).indices.int()      # [VOCAB][children]


class Server:
    """Caches and page table of a batch, and the buffers and plans of its steps."""

    def __init__(self, model, prompts, pages, table, seed=1):
        i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(device="cuda")
        self.m, self.P, self.Q, self.T = model, pages, len(prompts), len(TREE)
        Q, R = self.Q, self.Q * self.T
        self.R, self.max_ctx = R, table * lib.IDX_PAGE
        codes = lambda *shape: torch.zeros(pages, lib.IDX_PAGE, *shape, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.k, self.v, self.idx_k = codes(HKV, D), codes(HKV, D), codes(1, IDX_D)
        self.k_scale, self.v_scale, self.idx_scale = (torch.ones(pages, h, lib.IDX_PAGE, **f32) for h in (HKV, HKV, 1))
        self.cache = lib.make_kv_cache(self.k, self.v, self.k_scale, self.v_scale)
        self.idx_cache = lib.make_kv_cache(self.idx_k, None, self.idx_scale, None)
        self.page_table = torch.full((Q, table), -1, **i32)
        self.free_pages = torch.arange(pages, **i32).flip(0).contiguous()
        self.free_count = torch.full((1,), pages, **i32)
        self.free_left = torch.zeros(1, **i32)
        self.ctx = torch.zeros(Q, **i32)
        self.tables_state = lib.alloc_state(lib.tree_tables_state_size())

        # the prompts but for their last tokens, which the first step starts with
        self.prompt(prompts)

        # a step
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.token0 = torch.tensor([int(p[-1]) for p in prompts], **i32)
        self.new_len = torch.full((Q,), self.T, **i32)
        self.parent = torch.tensor(TREE * Q, **i32)
        self.rank = torch.tensor([TREE[:n].count(p) for n, p in enumerate(TREE)])   # which child of its parent
        self.draft, self.target, self.path, self.token, self.accept_len, self.last = (torch.zeros(n, **i32) for n in (R, R, R, R, Q, Q))
        self.logprob, self.u = torch.zeros(R, **f32), torch.zeros(R, **f32)
        each = lambda values, dtype: torch.tensor([values[i % len(values)] for i in range(Q) for _ in TREE], dtype=dtype, device="cuda")  # noqa: E731
        self.temperature, self.top_k = each((0.0, 0.7, 1.0, 0.5), torch.float32), each((0, 40, 0, 100), torch.int32)
        self.top_p, self.min_p = each((1.0, 1.0, 0.9, 0.95), torch.float32), each((0.0, 0.0, 0.0, 0.02), torch.float32)
        self.rows = self.row_buffers(R)
        self.q, self.idx_q, self.out = (torch.zeros(R, *d, dtype=torch.bfloat16, device="cuda") for d in ((HQ, D), (IDX_HEADS, IDX_D), (HQ, D)))
        self.idx_w, self.logits = torch.zeros(R, IDX_HEADS, **f32), torch.zeros(R, VOCAB, **f32)
        self.bound, self.sel = torch.zeros(R, **i32), torch.zeros(R, K, **i32)
        self.ranked = lib.make_problem(self.idx_q, self.idx_w, self.idx_k.squeeze(2), self.idx_scale.squeeze(1), self.page_table,
                                       self.rows["row_req"], self.bound, self.max_ctx, lib.IDX_KV_E4M3)
        self.attention = lib.make_tree_problem(self.q, self.cache, self.page_table, self.ctx, self.rows["row_start"], self.rows["mask"],
                                               self.max_ctx, self.T, D ** -0.5)
        self.ws = lib.alloc_bytes(lib.workspace_size(self.ranked, K))
        self.attention_state = lib.alloc_state(lib.tree_state_size(self.attention, K))
        self.sampling = lib.make_sample(self.logits, self.u, self.target, logprob=self.logprob, temperature=self.temperature,
                                        top_k=self.top_k, top_p=self.top_p, min_p=self.min_p)
        self.accept_state = lib.alloc_state(lib.tree_accept_state_size())
        self.acceptance = lib.make_tree_accept(self.rows["row_start"], self.draft, self.target, self.ctx, self.page_table,
                                               self.free_pages, self.free_left, P=self.P, new_ctx=self.ctx, accept_len=self.accept_len,
                                               last=self.last, path=self.path, token=self.token, free_left=self.free_count,
                                               parent=self.parent)

    def row_buffers(self, R):
        """What idx_tree_tables says of every row."""
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(row_start=torch.zeros(self.Q + 1, **i32), mask=torch.zeros(R, dtype=torch.int64, device="cuda"),
                    **{n: torch.zeros(R, **i32) for n in ("row_req", "row_bound", "row_pos", "slot")})

    def place(self, new_len, rows, parent):
        t = lib.make_tree_tables(self.ctx, new_len, self.page_table, self.free_pages, self.free_count, P=self.P, free_left=self.free_left,
                                 parent=parent, **dict(rows, mask=None if parent is None else rows["mask"]))
        lib.idx_tree_tables(t, self.tables_state)

    def prepare(self, tokens, pos, slot, cache, idx_cache, q=None, idx_q=None):
        """Keys and values of tokens [R] into the caches, queries into q and idx_q where they are wanted."""
        m = self.m
        qkv, idx_qk = m.qkv[tokens], m.idx_qk[tokens]
        lib.idx_norm_rope(lib.make_norm_rope(None if q is None else qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], q_out=q, pos=pos,
                                             inv_freq=m.inv_freq, cache=cache, slot=slot, k_weight=m.k_weight,
                                             q_weight=None if q is None else m.q_weight))
        lib.idx_norm_rope(lib.make_norm_rope(None if q is None else idx_qk[:, :IDX_HEADS], idx_qk[:, IDX_HEADS:], q_out=idx_q, pos=pos,
                                             inv_freq=m.idx_inv_freq, cache=idx_cache, slot=slot, interleaved=True,
                                             q_norm=lib.IDX_NORM_NONE, k_norm=lib.IDX_NORM_LAYER, k_weight=m.idx_k_weight,
                                             k_bias=m.idx_k_bias))

    def prompt(self, prompts):
        tokens = torch.cat([p[:-1] for p in prompts]).cuda().long()
        lens = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device="cuda")
        rows = self.row_buffers(tokens.numel())
        self.place(lens, rows, None)
        self.prepare(tokens, rows["row_pos"], rows["slot"], self.cache, self.idx_cache)
        self.ctx += lens
        self.free_count.copy_(self.free_left)

    def step(self):
        m, draft = self.m, self.draft.view(self.Q, self.T)
        draft[:, 0] = self.token0
        for n in range(1, self.T):
            draft[:, n] = m.likely[draft[:, TREE[n]].long(), int(self.rank[n])]
        tokens = self.draft.long()
        rows = self.rows
        self.place(self.new_len, rows, self.parent)
        self.prepare(tokens, rows["row_pos"], rows["slot"], self.cache, self.idx_cache, self.q, self.idx_q)

        self.idx_w.copy_(m.idx_w[tokens])
        self.bound.copy_(self.ctx[rows["row_req"].long()])      # every token ranks its request's cached positions
        lib.idx_launch(self.ranked, K, self.sel, self.ws)
        lib.idx_tree_attention_selected(self.attention, self.sel, self.out, self.attention_state)

        self.logits.copy_(self.out.flatten(1) @ m.out + m.skip[tokens])
        lib.idx_sample(self.sampling)
        lib.idx_tree_accept(self.acceptance, self.accept_state)
        for cache in (self.cache, self.idx_cache):
            lib.idx_tree_commit(cache, rows["row_start"], self.accept_len, self.path, rows["slot"])
        self.token0.copy_(self.last)

    def numbers(self):
        self.u.copy_(torch.rand(self.R, device="cuda", generator=self.gen))

    def captured(self):
        """The step as a graph, after one that ran."""
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def check(self):
        for name, st in (("tables", self.tables_state), ("attention", self.attention_state), ("acceptance", self.accept_state)):
            status = lib.last_device_status(st)
            if status != lib.IDX_OK:
                raise lib.IdxError(status, name)


def main(prompts=(3000, 1100, 64, 1), steps=12, graph=True, seed=1, each=None, verbose=True):
    """Runs `steps` steps; each(server) is called behind every one."""
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(VOCAB, (n,), generator=g) for n in prompts]
    pages = sum((len(p) + lib.IDX_PAGE - 2) // lib.IDX_PAGE + 1 for p in prompts) + len(prompts) * (1 + steps * len(TREE) // lib.IDX_PAGE)
    s = Server(Model(), prompts, pages, table=max(len(p) for p in prompts) // lib.IDX_PAGE + 2 + steps * len(TREE) // lib.IDX_PAGE, seed=seed)
    text = [p.tolist() for p in prompts]
    replay = None
    for n in range(steps):
        s.numbers()
        if n == 0 or not graph:
            s.step()
        else:
            replay = replay or s.captured()
            replay.replay()
        new, count = s.token.view(s.Q, s.T).tolist(), s.accept_len.tolist()
        for i in range(s.Q):
            text[i] += new[i][:count[i]]
        if each is not None:
            each(s)
    s.check()
    if verbose:
        for i, p in enumerate(prompts):
            print(f"request {i}: {len(text[i]) - len(p)} tokens in {steps} steps behind {len(p)}, {int(s.ctx[i])} cached: {text[i][len(p):]}")
    return s, text


if __name__ == "__main__":
    main()
