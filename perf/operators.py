"""The operators of a tree-verify decode step: cases, plain forms and exact values.

    tables    page tables, slot maps and tree masks of a step from request lengths
    write     new tokens' K and V into the paged cache, at their slots
    attend    attention of each request's drafted tokens (a tree) over its paged cache
    selected  the same over the positions that the indexer selected for each row

With ``own`` false, ``run`` computes an operator from elementary torch operations;
with ``own`` true it calls this repository's entry points.  Pages hold 64 tokens, and
the attention operators see a cached position j < ctx (all of them, or the selected
ones) and a drafted token u iff bit u of the row's mask is set.
"""
import random

import torch

own = False

PAGE = 64
DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # two long requests with a 4-token draft chain each: the smallest call, all latency
        dict(name="tables 2x4 at 512K", op="tables", Q=2, ctx_lo=524288, ctx_hi=524288, new_lo=4, new_hi=4, tree=False, shape=1),
        # a serving batch of drafted trees, some on a page's edge
        dict(name="tables 64 trees", op="tables", Q=64, ctx_lo=1024, ctx_hi=524288, new_lo=1, new_hi=64, tree=True, shape=2),
        # admission of 64 prompts: millions of slots
        dict(name="tables 64 prompts", op="tables", Q=64, ctx_lo=0, ctx_hi=0, new_lo=1024, new_hi=524288, tree=False, shape=3),
        # a verify step's 32 rows into a bf16 cache
        dict(name="write 8x4 bf16", op="write", Q=8, ctx_lo=8192, ctx_hi=65536, new_lo=4, new_hi=4, Hq=64, Hkv=8, D=128, kv="bf16", major="token", shape=4),
        # prompts into an E4M3 cache: quantised while they are written
        dict(name="write 64K e4m3", op="write", Q=9, ctx_lo=0, ctx_hi=0, new_lo=4096, new_hi=12287, Hq=64, Hkv=8, D=128, kv="e4m3", major="head", shape=5),
        # one token of one request at 4,096 keys: the latency of a lone decode row
        dict(name="attend 1x1 at 4K", op="attend", Q=1, ctx_lo=4095, ctx_hi=4095, new_lo=1, new_hi=1, Hq=64, Hkv=8, D=128, kv="bf16", major="token", shape=6),
        # one request's 4-token chain at 131,072 keys of an E4M3 cache
        dict(name="attend 1x4 at 128K e4m3", op="attend", Q=1, ctx_lo=131069, ctx_hi=131069, new_lo=4, new_hi=4, Hq=64, Hkv=8, D=128, kv="e4m3", major="head", shape=7),
        # eight requests' 16-node trees over 8K-256K keys: the cache's bandwidth
        dict(name="attend 8x16 to 256K", op="attend", Q=8, ctx_lo=8192, ctx_hi=262144, new_lo=16, new_hi=16, Hq=64, Hkv=8, D=128, kv="bf16", major="token", shape=8),
        # 64-node trees on one shared key head: all arithmetic
        dict(name="attend 4x64 one kv head", op="attend", Q=4, ctx_lo=12000, ctx_hi=30000, new_lo=64, new_hi=64, Hq=64, Hkv=1, D=128, kv="bf16", major="token", shape=9),
        # a ragged batch of short draft chains with small heads
        dict(name="attend 64x1-4 D64 e4m3", op="attend", Q=64, ctx_lo=1024, ctx_hi=32768, new_lo=1, new_hi=4, Hq=32, Hkv=8, D=64, kv="e4m3", major="token", shape=10),
        # the indexer's benchmark rows (2 requests x 4 rows at 512K) over their top 2,048
        dict(name="selected 2x4 at 512K", op="selected", Q=2, ctx_lo=524288, ctx_hi=524288, new_lo=4, new_hi=4, K=2048, Hq=64, Hkv=1, D=128, kv="bf16", major="token", shape=11),
        # a ragged batch of verify rows over their top 2,048 of an E4M3 cache
        dict(name="selected 64x1-4 e4m3", op="selected", Q=64, ctx_lo=1024, ctx_hi=65536, new_lo=1, new_hi=4, K=2048, Hq=64, Hkv=2, D=128, kv="e4m3", major="token", shape=12),
    ]


def _log(rng, lo, hi):
    """An integer of lo..hi, spread over its logarithm."""
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(max(lo, 1) * (hi / max(lo, 1)) ** rng.random()))))


def _lengths(c):
    """(ctx, new) of every request: the case's own numbers, whatever the seed."""
    rng = random.Random(1000 * c["shape"] + c["Q"])
    ctx = [_log(rng, c["ctx_lo"], c["ctx_hi"]) for _ in range(c["Q"])]
    new = [rng.randint(c["new_lo"], c["new_hi"]) if c["new_hi"] < 1024 else _log(rng, c["new_lo"], c["new_hi"]) for _ in range(c["Q"])]
    return ctx, new


def draw(rng):
    op = rng.choice(["tables", "write", "attend", "attend", "attend", "selected"])
    c = dict(op=op, shape=rng.randint(100, 1 << 20))
    while True:
        c["Q"] = _log(rng, 1, 64)
        lo, hi = sorted((_log(rng, 1, 300000), _log(rng, 1, 300000)))
        c["ctx_lo"], c["ctx_hi"] = lo, hi
        if op == "tables":
            c["tree"] = rng.random() < 0.5
            c["new_lo"], c["new_hi"] = sorted((_log(rng, 1, 64), _log(rng, 1, 64))) if c["tree"] or rng.random() < 0.5 else (lo, hi)
            ok = sum(_lengths(c)[1]) <= 4000000
        else:
            c["Hq"], c["Hkv"] = rng.choice([(64, 8), (64, 1), (32, 8), (16, 16), (64, 2), (24, 4), (8, 8)])
            c["D"] = rng.choice([64, 128, 128])
            c["kv"] = rng.choice(["bf16", "e4m3"])
            c["major"] = rng.choice(["token", "head"])
            if op == "write":
                if rng.random() < 0.5:
                    c["ctx_lo"] = c["ctx_hi"] = 0
                    c["new_lo"], c["new_hi"] = sorted((_log(rng, 100, 20000), _log(rng, 100, 20000)))
                else:
                    c["new_lo"], c["new_hi"] = sorted((_log(rng, 1, 64), _log(rng, 1, 64)))
                    c["ctx_lo"], c["ctx_hi"] = min(lo, 8192), min(hi, 16384)
                ctx, new = _lengths(c)
                # tokens written, and the cache that is returned whole
                ok = sum(new) <= 65000 and (sum(ctx) + sum(new)) * c["Hkv"] * c["D"] <= 2e8
            else:
                c["new_lo"], c["new_hi"] = sorted((_log(rng, 1, 64), _log(rng, 1, 64)))
                if op == "selected":
                    c["K"] = _log(rng, 64, 2048)
                    c["new_lo"], c["new_hi"] = min(c["new_lo"], 16), min(c["new_hi"], 16)
                ctx, new = _lengths(c)
                padded = c["Q"] * (max(ctx) + max(new)) * c["Hkv"]
                w = work(c)
                if op == "attend":
                    ok = (w["bytes"] <= 2.2e9 and w["flops"] <= 1.5e11 and padded * c["D"] <= 2.2e9 and c["Q"] * max(new) * c["Hq"] * (max(ctx) + max(new)) <= 2.3e9)
                else:
                    ok = (w["bytes"] <= 1.8e8 and w["flops"] <= 1.2e10 and (sum(ctx) + sum(new)) * c["Hkv"] * c["D"] <= 2.2e8)
        if ok:
            return c


def work(c):
    ctx, new = _lengths(c)
    R = sum(new)
    if c["op"] == "tables":
        pages = sum((a + n + 63) // 64 - (a + 63) // 64 for a, n in zip(ctx, new))
        per_row = 4 * 4 + (4 + 8 if c["tree"] else 0)
        return {"bytes": 12 * c["Q"] + 8 * pages + per_row * R, "flops": 0}
    e = 2 if c["kv"] == "bf16" else 1
    tok = c["Hkv"] * (2 * c["D"] * e + (8 if e == 1 else 0))     # one token's K and V, with scales
    if c["op"] == "write":
        return {"bytes": R * (4 * c["Hkv"] * c["D"] + tok + 4), "flops": 0}
    io = R * c["Hq"] * (4 * c["D"] + 4)
    if c["op"] == "attend":
        keys = sum(a + n for a, n in zip(ctx, new) if n)
        pairs = sum(n * a + _seen(c, n) for a, n in zip(ctx, new))
        return {"bytes": keys * tok + io, "flops": 4 * c["D"] * c["Hq"] * pairs}
    pairs = sum(n * min(c["K"], a) + _seen(c, n) for a, n in zip(ctx, new))
    # a position that several rows of one request select has to be read once
    keys = sum(min(n * min(c["K"], a), a) + n for a, n in zip(ctx, new))
    return {"bytes": keys * tok + io + 4 * R * c["K"], "flops": 4 * c["D"] * c["Hq"] * pairs}


def _seen(c, n):
    """Mask bits set in a tree of n nodes (node t's parent is (t - 1) // 2)."""
    return sum((t + 1).bit_length() for t in range(n))


# ---------------------------------------------------------------------------- inputs
def _parents(n):
    """A tree's parent list: node 0 the root, node t under (t - 1) // 2."""
    return [(t - 1) // 2 if t else -1 for t in range(n)]


def _masks(n):
    got = []
    for t, p in enumerate(_parents(n)):
        got.append((1 << t) | (got[p] if p >= 0 else 0))
    return [m - (1 << 64) if m >> 63 else m for m in got]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(new):
    got = [0]
    for n in new:
        got.append(got[-1] + n)
    return got


def _quantised(x):
    """E4M3 codes and one fp32 scale per last-dimension vector: amax / 448."""
    amax = x.float().abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x.float() / sc[..., None]).to(torch.float8_e4m3fn), sc


def _cache(c, P, gen):
    """K or V of P pages as [P][64][Hkv][D] (its memory token- or head-major), with scales [P][Hkv][64]."""
    if c["major"] == "token":
        x = torch.empty(P, PAGE, c["Hkv"], c["D"], dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    else:
        x = torch.empty(P, c["Hkv"], PAGE, c["D"], dtype=torch.bfloat16, device=DEV).normal_(generator=gen).transpose(1, 2)
    if c["kv"] == "bf16":
        return x, None
    code, sc = _quantised(x)            # strides of x are kept
    return code, sc.transpose(1, 2).contiguous()


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ctx, new = _lengths(c)
    Q, R = c["Q"], sum(new)
    start = _starts(new)
    pages = [(a + n + PAGE - 1) // PAGE for a, n in zip(ctx, new)]
    held = [(a + PAGE - 1) // PAGE for a in ctx]
    P = sum(pages) + 3
    stride = max(pages) + 1
    perm = torch.randperm(P, device=DEV, generator=gen).to(torch.int32)
    s = dict(case=c, R=R, P=P, ctx=_i32(ctx), new=_i32(new), max_ctx=max(ctx), max_new=max(new))
    # every request's pages: a random choice from one pool
    j = torch.arange(stride, device=DEV)[None]
    first = torch.tensor(_starts(pages)[:-1], device=DEV)[:, None]
    have = torch.tensor(held if c["op"] == "tables" else pages, device=DEV)[:, None]
    s["page_table"] = torch.where(j < have, perm[(first + j).clamp(max=P - 1)], -1).to(torch.int32)

    if c["op"] == "tables":
        cap = (R + 7) // 8 * 8
        s["cap"], s["take"] = cap, sum(pages) - sum(held)
        # the free stack: the pages that no request holds
        gone = torch.zeros(P, dtype=torch.bool, device=DEV)
        gone[s["page_table"][s["page_table"] >= 0].long()] = True
        s["free"] = perm[~gone[perm.long()]].contiguous()
        s["free_count"] = _i32([s["free"].numel()])
        s["parent"] = _i32(sum((_parents(n) for n in new), []) + [-1] * (cap - R)) if c["tree"] else None
        if own:
            import sparse_attention_indexer_launch_gb300 as lib
            o = s["o"] = dict(row_start=torch.empty(Q + 1, dtype=torch.int32, device=DEV), free_left=torch.empty(1, dtype=torch.int32, device=DEV))
            for k in ("row_req", "row_bound", "row_pos", "slot"):
                o[k] = torch.empty(cap, dtype=torch.int32, device=DEV)
            o["mask"] = torch.empty(cap, dtype=torch.int64, device=DEV) if c["tree"] else None
            s["plan"] = lib.make_tree_tables(s["ctx"], s["new"], s["page_table"], s["free"], s["free_count"], parent=s["parent"], P=P, **o)
            s["ws"] = lib.alloc_state(lib.tree_tables_state_size())
        return s

    s["row_start"] = _i32(start)
    s["row_req"] = torch.repeat_interleave(torch.arange(Q, device=DEV), s["new"].long(), output_size=R)
    s["t"] = torch.arange(R, device=DEV) - s["row_start"].long()[s["row_req"]]
    s["mask"] = torch.tensor(sum((_masks(n) for n in new), []) if c["op"] != "write" else [0], dtype=torch.int64, device=DEV)
    s["k"], s["k_scale"] = _cache(c, P, gen)
    s["v"], s["v_scale"] = _cache(c, P, gen)
    # queries, keys and values as one projection leaves them: [R][Hq + 2 Hkv][D]
    qkv = torch.empty(R, c["Hq"] + 2 * c["Hkv"], c["D"], dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    s["q"] = qkv[:, :c["Hq"]].mul_(2.0)
    s["k_new"], s["v_new"] = qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], qkv[:, c["Hq"] + c["Hkv"]:]
    at = s["ctx"].long()[s["row_req"]] + s["t"]
    s["slot"] = (s["page_table"][s["row_req"], at // PAGE] * PAGE + (at % PAGE)).to(torch.int32)
    if c["op"] == "selected":
        s["sel"] = torch.full((R, c["K"]), -1, dtype=torch.int32, device=DEV)
        for r in range(R):
            a = ctx[int(r_of(start, r))]
            if a:
                got = torch.rand(a, device=DEV, generator=gen).topk(min(c["K"], a)).indices
                s["sel"][r, :got.numel()] = got.to(torch.int32)
    if own:
        import sparse_attention_indexer_launch_gb300 as lib
        s["cache"] = lib.make_kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if c["op"] != "write":
            s["plan"] = lib.make_tree_problem(s["q"], s["cache"], s["page_table"], s["ctx"], s["row_start"], s["mask"], s["max_ctx"], s["max_new"], c["D"] ** -0.5)
            s["out"] = torch.empty(R, c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(R, c["Hq"], dtype=torch.float32, device=DEV)
            s["ws"] = lib.alloc_state(lib.tree_state_size(s["plan"], c.get("K", 0)))
    return s


def r_of(start, r):
    """The request of row r."""
    lo, hi = 0, len(start) - 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if start[mid] <= r else (lo, mid)
    return lo


# ---------------------------------------------------------------------------- run
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_launch_gb300 as lib
    op = s["case"]["op"]
    if op == "tables":
        lib.idx_tree_tables(s["plan"], s["ws"])
        return dict(s["o"], page_table=s["page_table"])
    if op == "write":
        lib.idx_write_kv(s["cache"], s["k_new"], s["v_new"], s["slot"])
        return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "attend":
        lib.idx_tree_attention(s["plan"], s["out"], s["ws"], lse=s["lse"])
    else:
        lib.idx_tree_attention_selected(s["plan"], s["sel"], s["out"], s["ws"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _run_plain(s):
    return dict(tables=_plain_tables, write=_plain_write, attend=_plain_attend, selected=_plain_selected)[s["case"]["op"]](s)


def _plain_tables(s):
    ctx, new, R, cap = s["ctx"].long(), s["new"].long(), s["R"], s["cap"]
    Q = ctx.numel()
    held = (ctx + PAGE - 1) // PAGE
    need = (ctx + new + PAGE - 1) // PAGE - held
    before = need.cumsum(0) - need
    count = s["free_count"].long()
    # new pages, from the top of the free stack
    i = torch.repeat_interleave(torch.arange(Q, device=DEV), need, output_size=s["take"])
    n = torch.arange(s["take"], device=DEV)
    s["page_table"][i, held[i] + n - before[i]] = s["free"][count - 1 - n]
    row_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    # rows
    req = torch.repeat_interleave(torch.arange(Q, device=DEV), new, output_size=R)
    t = torch.arange(R, device=DEV) - row_start[req]
    at = ctx[req] + t
    slot = s["page_table"][req, at // PAGE].long() * PAGE + at % PAGE
    depth, mask = t, None
    if s["parent"] is not None:
        # ancestors by doubling: after six steps every path of at most 64 nodes is closed
        par = s["parent"][:R].long()
        sees = torch.zeros(R, 64, dtype=torch.bool, device=DEV)
        sees[torch.arange(R, device=DEV), t] = True
        up = torch.where(par >= 0, row_start[req] + par, -1)
        for _ in range(6):
            sees = sees | (sees[up.clamp(min=0)] & (up >= 0)[:, None])
            up = torch.where(up >= 0, up[up.clamp(min=0)], -1)
        depth = sees.sum(1) - 1
        bits = torch.ones(64, dtype=torch.int64, device=DEV) << torch.arange(64, device=DEV)
        mask = _padded((sees * bits).sum(1), cap, 0)
    return dict(row_start=row_start.int(), free_left=(count - need.sum()).int(), row_req=_padded(req.int(), cap, 0), row_bound=_padded((at + 1).int(), cap, 0),
                row_pos=_padded((ctx[req] + depth).int(), cap, 0), slot=_padded(slot.int(), cap, -1), mask=mask, page_table=s["page_table"])


def _padded(x, n, value):
    return torch.cat([x, x.new_full((n - x.numel(),), value)])


def _plain_write(s):
    page, off = s["slot"].long() // PAGE, s["slot"].long() % PAGE
    if s["case"]["kv"] == "bf16":
        s["k"][page, off], s["v"][page, off] = s["k_new"], s["v_new"]
    else:
        code, sc = _quantised(s["k_new"])
        s["k"].view(torch.uint8)[page, off], s["k_scale"][page, :, off] = code.view(torch.uint8), sc
        code, sc = _quantised(s["v_new"])
        s["v"].view(torch.uint8)[page, off], s["v_scale"][page, :, off] = code.view(torch.uint8), sc
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _gathered(x, scale, page, off):
    """Tokens of the cache in fp32: [..., Hkv, D] at (page, off) of any shape."""
    if scale is None:
        return x[page, off].float()
    return x.view(torch.uint8)[page, off].view(torch.float8_e4m3fn).float() * scale[page, :, off][..., None]


def _softmax_times(score, visible, v):
    """(softmax over the visible keys) v, and log sum exp; zeros and -inf where nothing is visible."""
    score = score.masked_fill_(~visible, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return out, (l.log() + top)[..., 0]


def _plain_attend(s):
    c = s["case"]
    Hq, Hkv, D, Q = c["Hq"], c["Hkv"], c["D"], c["Q"]
    G, T, ctx = Hq // Hkv, s["max_new"], s["ctx"].long()
    S = s["max_ctx"] + T
    j = torch.arange(S, device=DEV)
    page = s["page_table"][:, (j // PAGE).clamp(max=s["page_table"].shape[1] - 1)].clamp(min=0).long()
    off = (j % PAGE).expand(Q, S)
    # requests' rows padded to [Q][T]
    row = (s["row_start"][:-1].long()[:, None] + torch.arange(T, device=DEV)).clamp(max=max(s["R"] - 1, 0))
    q = s["q"][row].float().view(Q, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(Q, Hkv, T * G, D)
    k = _gathered(s["k"], s["k_scale"], page, off)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5)
    del k
    u = j[None] - ctx[:, None]
    bit = (s["mask"][row][:, :, None] >> u.clamp(0, 63)[:, None]) & 1
    visible = (u < 0)[:, None] | ((u >= 0) & (u < s["new"][:, None]))[:, None] & (bit == 1)
    visible = visible[:, None, :, None].expand(Q, 1, T, G, S).reshape(Q, 1, T * G, S)
    v = _gathered(s["v"], s["v_scale"], page, off)
    out, lse = _softmax_times(score, visible, v.permute(0, 2, 1, 3))
    out = out.view(Q, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(Q, T, Hq, D)[s["row_req"], s["t"]]
    lse = lse.view(Q, Hkv, T, G).permute(0, 2, 1, 3).reshape(Q, T, Hq)[s["row_req"], s["t"]]
    return dict(out=out.bfloat16(), lse=lse)


def _plain_selected(s):
    c = s["case"]
    Hq, Hkv, D, R = c["Hq"], c["Hkv"], c["D"], s["R"]
    req, T = s["row_req"], s["max_new"]
    ctx = s["ctx"].long()[req]
    sel = s["sel"].long()
    u = torch.arange(T, device=DEV)
    at = torch.cat([sel.clamp(min=0), ctx[:, None] + u], 1)
    visible = torch.cat([(sel >= 0) & (sel < ctx[:, None]), ((s["mask"][:, None] >> u) & 1) == 1], 1)
    page = s["page_table"][req[:, None], (at // PAGE).clamp(max=s["page_table"].shape[1] - 1)].clamp(min=0).long()
    off = at % PAGE
    q = s["q"].float().view(R, Hkv, Hq // Hkv, D)
    k = _gathered(s["k"], s["k_scale"], page, off)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5)
    v = _gathered(s["v"], s["v_scale"], page, off)
    out, lse = _softmax_times(score, visible[:, None, None, :], v.permute(0, 2, 1, 3))
    return dict(out=out.reshape(R, Hq, D).bfloat16(), lse=lse.reshape(R, Hq))


# ---------------------------------------------------------------------------- 64 bits
def _e4m3_exact(x):
    """Nearest E4M3 value (ties to even) of float64 x with |x| <= 448."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(c, seed):
    if c["op"] == "tables":
        return None                       # whole numbers only
    s = prepare(c, seed)
    ctx, new = _lengths(c)
    start = _starts(new)
    table = s["page_table"].long()
    if c["op"] == "write":
        got = {}
        for name in ("k", "v"):
            x = s[name + "_new"].double()
            page, off = s["slot"].long() // PAGE, s["slot"].long() % PAGE
            if c["kv"] == "bf16":
                full = s[name].double()
                full[page, off] = x
                got[name], got[name + "_scale"] = full, None
            else:
                amax = x.abs().amax(-1)
                sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
                full = s[name].double()
                full[page, off] = _e4m3_exact(x / sc[..., None])
                scale = s[name + "_scale"].double()
                scale[page, :, off] = sc
                got[name], got[name + "_scale"] = full, scale
        return got
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.zeros(s["R"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((s["R"], Hq), float("-inf"), dtype=torch.float64, device=DEV)

    def tokens(i, at, h):
        page, off = table[i, at // PAGE], at % PAGE
        kv = []
        for name in ("k", "v"):
            x = s[name][:, :, h].reshape(-1, D)[page * PAGE + off].double() if c["kv"] == "bf16" else \
                s[name].view(torch.uint8)[page, off, h].view(torch.float8_e4m3fn).double()
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"][page, h, off].double()[:, None]
            kv.append(x)
        return kv

    def attend(rows, at, seen, i):
        """rows over the positions `at` of request i; seen: [rows][positions]."""
        for h in range(Hkv):
            k, v = tokens(i, at, h)
            q = s["q"][rows, h * G:(h + 1) * G].double()
            x = torch.einsum("rgd,sd->rgs", q, k) / D ** 0.5
            x = torch.where(seen[:, None], x, float("-inf"))
            z = torch.logsumexp(x, -1)
            out[rows, h * G:(h + 1) * G] = torch.einsum("rgs,sd->rgd", torch.exp(x - z[..., None]), v)
            lse[rows, h * G:(h + 1) * G] = z

    for i in range(c["Q"]):
        bits = torch.tensor([[(m >> u) & 1 for u in range(new[i])] for m in _masks(new[i])], dtype=torch.bool, device=DEV).view(new[i], new[i])
        drafted = ctx[i] + torch.arange(new[i], device=DEV)
        if c["op"] == "attend":
            # a few rows at a time: at most 16 x Hq / Hkv vectors against every key
            at = torch.arange(ctx[i] + new[i], device=DEV)
            for t in range(0, new[i], 16):
                b = bits[t:t + 16]
                seen = torch.cat([torch.ones(b.shape[0], ctx[i], dtype=torch.bool, device=DEV), b], 1)
                attend(torch.arange(start[i] + t, start[i] + t + b.shape[0], device=DEV), at, seen, i)
        else:
            for t in range(new[i]):
                sel = s["sel"][start[i] + t].long()
                sel = sel[sel >= 0]
                at = torch.cat([sel, drafted[bits[t]]])
                attend(torch.tensor([start[i] + t], device=DEV), at, torch.ones(1, at.numel(), dtype=torch.bool, device=DEV), i)
    return dict(out=out, lse=lse)
