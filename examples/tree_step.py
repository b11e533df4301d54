"""One verify step over drafted trees, with every call of the library that it takes.

A batch of requests has prompts in a paged cache (keys and values of the model, and the
indexer's keys, under one page table).  A step then
  1. gives the drafted tokens their pages, slots and tree masks    idx_tree_tables
  2. writes their keys and values                                  idx_write_kv
     and their indexer keys                                        idx_patch_new_keys
  3. ranks the cached positions for every drafted token            idx_launch
  4. attends to the selected positions and the token's ancestors   idx_tree_attention_selected
  5. takes the next token of every row                             idx_top1
The weights are random; the shapes are those of a model with 16 query heads, 2 key/value
heads of dimension 128 and an E4M3 cache.  Needs a GB300.

    python examples/tree_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_launch_gb300 as lib  # noqa: E402

HQ, HKV, D, IDX_HEADS, K, VOCAB = 16, 2, 128, 64, 2048, 32000


class Serving:
    """Caches, page table and free pages of a batch, and the buffers of its steps."""

    def __init__(self, Q, pages, table, rows, seed=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        u8 = dict(dtype=torch.uint8, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.P, self.Q = pages, Q
        self.k, self.v = (torch.zeros(pages, lib.IDX_PAGE, HKV, D, **u8) for _ in "kv")
        self.k_scale, self.v_scale = (torch.ones(pages, HKV, lib.IDX_PAGE, device="cuda") for _ in "kv")
        self.cache = lib.make_kv_cache(self.k, self.v, self.k_scale, self.v_scale)
        self.idx_k = torch.zeros(pages, lib.IDX_PAGE, 128, **u8)
        self.idx_scale = torch.ones(pages, lib.IDX_PAGE, device="cuda")
        self.page_table = torch.full((Q, table), -1, **i32)
        self.free_pages = torch.arange(pages, **i32).flip(0).contiguous()   # page 0 on top
        self.free_count = torch.full((1,), pages, **i32)
        self.free_left = torch.zeros(1, **i32)
        self.ctx = torch.zeros(Q, **i32)
        self.rows = rows
        self.row_start = torch.zeros(Q + 1, **i32)
        self.row_req, self.row_bound, self.row_pos, self.slot = (torch.zeros(rows, **i32) for _ in range(4))
        self.mask = torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.tables_state = lib.alloc_state(lib.tree_tables_state_size())

    def place(self, new_len, parent=None):
        """Pages and slots for new_len [Q] tokens; with parents also their tree masks."""
        t = lib.make_tree_tables(self.ctx, new_len, self.page_table, self.free_pages, self.free_count, P=self.P,
                                 row_start=self.row_start, free_left=self.free_left, row_req=self.row_req,
                                 row_bound=self.row_bound, row_pos=self.row_pos, slot=self.slot,
                                 mask=None if parent is None else self.mask, parent=parent)
        lib.idx_tree_tables(t, self.tables_state)

    def index_problem(self, q, w, R, bound, max_bound):
        return lib.make_problem(q, w, self.idx_k, self.idx_scale, self.page_table, self.row_req[:R], bound, max_bound,
                                lib.IDX_KV_E4M3)

    def random(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.gen).bfloat16()

    def write(self, R, max_bound):
        """K, V and indexer keys of the placed tokens (random, as a model's projections would give them)."""
        qkv = self.random(R, HQ + 2 * HKV, D)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        lib.idx_write_kv(self.cache, k, v, self.slot[:R])
        iq, iw = self.random(R, IDX_HEADS, 128), torch.rand(R, IDX_HEADS, device="cuda", generator=self.gen)
        lib.idx_patch_new_keys(self.index_problem(iq, iw, R, self.row_bound[:R], max_bound), self.random(R, 128))
        return q, iq, iw

    def commit(self, new_len):
        """Keeps the placed tokens: their pages leave the free stack."""
        self.ctx += new_len
        self.free_count.copy_(self.free_left)


def main(prompts=(3000, 1100, 64, 700), tree=((-1, 0, 0, 1, 1, 2, 2, 3), (-1, 0, 1, 2), (-1,), (-1, 0, 0, 0, 1, 4)),
         verbose=True):
    Q, new = len(prompts), [len(t) for t in tree]
    R = sum(new)
    s = Serving(Q, pages=200, table=128, rows=sum(prompts))

    # the prompts: chains without masks
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    s.place(lens)
    s.write(sum(prompts), max(prompts))
    s.commit(lens)

    # the step
    new_len = torch.tensor(new, dtype=torch.int32, device="cuda")
    parent = torch.full((s.rows,), -1, dtype=torch.int32, device="cuda")
    parent[:R] = torch.tensor(sum((list(t) for t in tree), []), dtype=torch.int32)
    s.place(new_len, parent)
    max_ctx = max(prompts)
    q, iq, iw = s.write(R, max_ctx + max(new))

    bound = s.ctx[s.row_req[:R].long()]      # every drafted token ranks its request's cached positions
    ranked = s.index_problem(iq, iw, R, bound, max_ctx)
    sel = torch.empty(R, K, dtype=torch.int32, device="cuda")
    ws = lib.alloc_bytes(lib.workspace_size(ranked, K))
    lib.idx_launch(ranked, K, sel, ws)

    p = lib.make_tree_problem(q, s.cache, s.page_table, s.ctx, s.row_start, s.mask[:R], max_ctx, max(new), D ** -0.5)
    out, lse = torch.empty(R, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(R, HQ, device="cuda")
    state = lib.alloc_state(lib.tree_state_size(p, K))
    lib.idx_tree_attention_selected(p, sel, out, state, lse=lse)

    head = s.random(HQ * D, VOCAB) * (HQ * D) ** -0.5
    logits = (out.flatten(1) @ head).float()
    token = torch.empty(R, dtype=torch.int32, device="cuda")
    lib.idx_top1(logits, token, lib.alloc_state(lib.top1_state_size(R)))

    for name, st in (("tables", s.tables_state), ("attention", state)):
        status = lib.last_device_status(st)
        if status != lib.IDX_OK:
            raise lib.IdxError(status, name)
    if verbose:
        for i in range(Q):
            a, b = int(s.row_start[i]), int(s.row_start[i + 1])
            print(f"request {i}: {prompts[i]} cached, {b - a} drafted, next tokens {token[a:b].tolist()}")
    return dict(step=s, problem=p, sel=sel, out=out, lse=lse, logits=logits, token=token, R=R, prompts=prompts, new=new)


if __name__ == "__main__":
    main()
