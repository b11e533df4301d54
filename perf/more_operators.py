"""The operators at both ends of a verify step: cases, plain forms and exact values.

    prepare  norms of queries and keys for each head and the rotation to their positions,
             keys and values into the paged cache in the same pass
    sample   a token of every row of logits: temperature, top-k, top-p, min-p, from
             given random numbers
    accept   the drafted tokens of every tree that the sampled ones confirm, and the
             pages behind them back on the free stack
    commit   the accepted tokens' keys and values to consecutive positions

With ``own`` false, ``run`` computes an operator from elementary torch operations;
with ``own`` true it calls this repository's entry points.  Pages hold 64 tokens.
"""
import random

import torch

own = False

PAGE = 64
DEV = "cuda"
EPS = 1e-6
FAR = 524288


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # two long requests with a 4-token draft chain each, at the benchmark's context: all latency
        dict(name="prepare 2x4 bf16", op="prepare", R=8, Hq=64, Hkv=8, D=128, kv="bf16", norm="rms", k_norm="rms", rot=128, pairs="halves", axes=1, run=4, shape=1),
        # the indexer's own queries and key: no norm and a LayerNorm, half of the dimensions rotated, keys alone cached
        dict(name="prepare indexer 160 rows", op="prepare", R=160, Hq=64, Hkv=1, D=128, kv="e4m3 keys", norm="none", k_norm="layer", rot=64, pairs="interleaved", axes=1, run=3, shape=2),
        # tokens of a video: time, height and width on three sections of the frequencies
        dict(name="prepare video 8855", op="prepare", R=8855, Hq=16, Hkv=16, D=128, kv="bf16", norm="rms", k_norm="rms", rot=128, pairs="halves", axes=3, run=8855, shape=3),
        # prompts into an E4M3 cache: quantised as they are written
        dict(name="prepare prompts 16K e4m3", op="prepare", R=16209, Hq=64, Hkv=8, D=128, kv="e4m3", norm="rms", k_norm="rms", rot=128, pairs="halves", axes=1, run=5403, shape=4),
        # one row of a small vocabulary: the latency of a lone decode row
        dict(name="sample 1x32000", op="sample", R=1, V=32000, dtype="fp32", temp=True, top_k=0, top_p=True, min_p=False, shape=5),
        # the verify rows of the benchmark's top-1 with every filter
        dict(name="sample 8x151552", op="sample", R=8, V=151552, dtype="fp32", temp=True, top_k=50, top_p=True, min_p=True, shape=6),
        # a batch of bf16 logits over the whole vocabulary: no filter
        dict(name="sample 64x128000 bf16", op="sample", R=64, V=128000, dtype="bf16", temp=True, top_k=0, top_p=False, min_p=False, shape=7),
        # a large batch, the nucleus of the whole vocabulary
        dict(name="sample 256x151552", op="sample", R=256, V=151552, dtype="fp32", temp=True, top_k=0, top_p=True, min_p=False, shape=8),
        # two 4-token chains, the smallest step
        dict(name="accept 2x4", op="accept", Q=2, new_lo=4, new_hi=4, tree=False, hit=0.7, shape=9),
        # many trees of up to 64 tokens
        dict(name="accept 1024 trees", op="accept", Q=1024, new_lo=1, new_hi=64, tree=True, hit=0.6, shape=10),
        # eight 16-node trees over a bf16 cache
        dict(name="commit 8x16 bf16", op="commit", Q=8, new_lo=16, new_hi=16, Hkv=8, D=128, kv="bf16", major="token", hit=0.8, shape=11),
        # a large ragged batch over an E4M3 cache, long accepted paths
        dict(name="commit 512x1-64 e4m3", op="commit", Q=512, new_lo=1, new_hi=64, Hkv=8, D=128, kv="e4m3", major="head", hit=1.0, shape=12),
    ]


def _log(rng, lo, hi):
    """An integer of lo..hi, spread over its logarithm."""
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _new(c):
    """Drafted tokens of every request: the case's own numbers, whatever the seed."""
    rng = random.Random(1000 * c["shape"] + c["Q"])
    return [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["Q"])]


def draw(rng):
    op = rng.choice(["prepare", "prepare", "sample", "sample", "sample", "accept", "commit"])
    c = dict(op=op, shape=rng.randint(100, 1 << 20))
    if op == "prepare":
        while True:
            c["R"] = _log(rng, 1, 30000)
            c["Hq"], c["Hkv"] = rng.choice([(64, 8), (64, 1), (32, 8), (16, 16), (24, 4), (5, 5), (8, 2)])
            c["D"] = rng.choice([64, 128, 128, 256])
            c["kv"] = rng.choice(["none", "bf16", "e4m3", "e4m3 keys"]) if c["D"] < 256 else "none"
            c["norm"] = rng.choice(["rms", "rms", "none", "layer"])
            c["k_norm"] = rng.choice([c["norm"], "rms", "layer"])
            c["rot"] = rng.choice([c["D"], c["D"], c["D"] // 2, c["D"] // 4])
            c["pairs"] = rng.choice(["halves", "interleaved"])
            c["axes"] = rng.choice([1, 1, 3])
            c["run"] = _log(rng, 1, c["R"])
            if c["R"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"] <= 16209 * 80 * 128:
                return c
    if op == "sample":
        while True:
            c["R"], c["V"] = _log(rng, 1, 256), _log(rng, 1000, 262144)
            c["dtype"] = rng.choice(["fp32", "bf16"])
            c["temp"], c["top_p"], c["min_p"] = rng.random() < 0.8, rng.random() < 0.5, rng.random() < 0.3
            c["top_k"] = rng.choice([0, 0, _log(rng, 1, 1000)])
            if c["R"] * c["V"] <= 256 * 151552:
                return c
    c["Q"] = _log(rng, 1, 1024 if op == "accept" else 512)
    c["new_lo"], c["new_hi"] = sorted((_log(rng, 1, 64), _log(rng, 1, 64)))
    c["hit"] = rng.choice([0.3, 0.6, 0.8, 1.0])
    if op == "accept":
        c["tree"] = rng.random() < 0.7
        return c
    c["Hkv"], c["D"] = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    c["kv"], c["major"] = rng.choice(["bf16", "e4m3"]), rng.choice(["token", "head"])
    return c


def work(c):
    if c["op"] == "prepare":
        q, kv = c["R"] * c["Hq"] * c["D"], c["R"] * c["Hkv"] * c["D"]
        n = 4 * q + 4 * c["R"] * c["axes"]
        if c["kv"] == "none":
            n += 4 * kv
        elif c["kv"] == "bf16":
            n += 8 * kv + 4 * c["R"]
        else:
            n += (2 if c["kv"] == "e4m3" else 1) * (3 * kv + 4 * c["R"] * c["Hkv"]) + 4 * c["R"]
        return {"bytes": n, "flops": 10 * (q + kv)}
    if c["op"] == "sample":
        return {"bytes": c["R"] * (c["V"] * (4 if c["dtype"] == "fp32" else 2) + 28), "flops": 0}
    R = sum(_new(c))
    if c["op"] == "accept":
        return {"bytes": R * (16 + (4 if c["tree"] else 0)) + 16 * c["Q"], "flops": 0}
    # a path of a tree of n nodes has at most log2 n moves; a token's K and V are read and written
    moved = sum(max(0, (n + 1).bit_length() - 2) for n in _new(c))
    tok = 2 * c["Hkv"] * (c["D"] * 2 if c["kv"] == "bf16" else c["D"] + 4)
    return {"bytes": 2 * moved * tok + 8 * R + 8 * c["Q"], "flops": 0}


# ---------------------------------------------------------------------------- inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rand(gen, *n):
    return torch.rand(*n, device=DEV, generator=gen)


def _quantised(x):
    """E4M3 codes and one fp32 scale per last-dimension vector: amax / 448."""
    amax = x.float().abs().amax(-1)
    sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x.float() / sc[..., None]).to(torch.float8_e4m3fn), sc


def _cache(c, P, gen):
    """K or V of P pages as [P][64][Hkv][D] (its memory token- or head-major), with scales [P][Hkv][64]."""
    if c.get("major", "token") == "token":
        x = torch.empty(P, PAGE, c["Hkv"], c["D"], dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    else:
        x = torch.empty(P, c["Hkv"], PAGE, c["D"], dtype=torch.bfloat16, device=DEV).normal_(generator=gen).transpose(1, 2)
    if c["kv"] == "bf16":
        return x, None
    code, sc = _quantised(x)            # strides of x are kept
    return code, sc.transpose(1, 2).contiguous()


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(prepare=_inputs_prepare, sample=_inputs_sample, accept=_inputs_accept, commit=_inputs_accept)[c["op"]](c, gen)
    s["case"] = c
    if own:
        _plan(s)
    return s


def _inputs_prepare(c, gen):
    R, Hq, Hkv, D, rot = (c[k] for k in ("R", "Hq", "Hkv", "D", "rot"))
    s = {}
    # queries, keys and values as one projection leaves them: [R][Hq + 2 Hkv][D], some rows louder than others
    x = torch.empty(R, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    x.mul_(torch.exp(_rand(gen, R, 1, 1) * 4 - 2))
    s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    for n in ("q", "k"):
        kind = c["norm"] if n == "q" else c["k_norm"]
        s[n + "_weight"] = None if kind == "none" else 0.5 + _rand(gen, D)
        s[n + "_bias"] = _rand(gen, D) - 0.5 if kind == "layer" else None
    s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).float()
    # consecutive positions in runs that start anywhere; with three axes a run is a video of 16 x 22 patches a frame
    r = torch.arange(R, device=DEV)
    first = (_rand(gen, (R + c["run"] - 1) // c["run"]) * (FAR - 1)).long()[r // c["run"]]
    at = r % c["run"]
    pos = first + at if c["axes"] == 1 else torch.stack([first + at // 352, first + at % 352 // 22, first + at % 22])
    s["pos"] = pos.to(torch.int32).view(c["axes"], R).contiguous()
    # the first quarter of the frequencies is the time's, the others are the height's and the width's
    n, k = rot // 2, rot // 8
    s["axis"] = [0] * n if c["axes"] == 1 else [0] * k + [1] * ((n - k + 1) // 2) + [2] * ((n - k) // 2)
    s["axis_of"] = torch.tensor(s["axis"], device=DEV)
    s["q_out"] = torch.empty(R, Hq, D, dtype=torch.bfloat16, device=DEV)
    s["k_out"] = torch.empty(R, Hkv, D, dtype=torch.bfloat16, device=DEV) if c["kv"] == "none" else None
    if c["kv"] != "none":
        P = (R + PAGE - 1) // PAGE + 3
        s["keys"], s["keys_scale"] = _cache(c, P, gen)
        s["values"], s["values_scale"] = (None, None) if c["kv"] == "e4m3 keys" else _cache(c, P, gen)
        page = torch.randperm(P, device=DEV, generator=gen)
        s["slot"] = (page[r // PAGE] * PAGE + r % PAGE).to(torch.int32)
    return s


def _inputs_sample(c, gen):
    R, V = c["R"], c["V"]
    # rows from flat to peaked; the last columns pad the vocabulary and are masked
    x = torch.empty(R, V, dtype=torch.float32, device=DEV).normal_(generator=gen)
    x.mul_(1 + 3 * _rand(gen, R, 1))
    x[:, V - V // 200:] = float("-inf")
    s = dict(logits=x if c["dtype"] == "fp32" else x.bfloat16(), u=_rand(gen, R))
    # a batch of many users: a tenth of them greedy, filters of various strength, some with none
    greedy, off = _rand(gen, R) < 0.1, _rand(gen, R) < 0.1
    s["temperature"] = torch.where(greedy, 0.0, 0.6 + 0.7 * _rand(gen, R)) if c["temp"] else None
    k = (c["top_k"] * (0.5 + _rand(gen, R))).long().clamp(min=1)
    s["top_k"] = torch.where(off, 0, k).to(torch.int32) if c["top_k"] else None
    s["top_p"] = torch.where(off, 1.0, 0.5 + 0.49 * _rand(gen, R)) if c["top_p"] else None
    s["min_p"] = torch.where(off, 0.0, 0.002 + 0.1 * _rand(gen, R)) if c["min_p"] else None
    return s


def _inputs_accept(c, gen):
    """Trees whose node t is under (t - 1) // 2, or chains; the sampled token is a child's draft with chance `hit`."""
    new = _new(c)
    Q, R = c["Q"], sum(new)
    tree = c["op"] == "commit" or c["tree"]
    s = dict(R=R)
    n = _i32(new).long()
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    s["row_start"] = start.to(torch.int32)
    s["req"] = torch.repeat_interleave(torch.arange(Q, device=DEV), n, output_size=R)
    s["t"] = t = torch.arange(R, device=DEV) - start[s["req"]]
    parent = torch.where(t > 0, (t - 1) // 2 if tree else t - 1, -1)
    s["parent"] = parent.to(torch.int32) if tree else None
    s["draft"] = (_rand(gen, R) * 150000).to(torch.int32)
    child = (2 * t + 1 + (_rand(gen, R) < 0.5)) if tree else t + 1
    have = (child < n[s["req"]]) & (_rand(gen, R) < c["hit"])
    other = (_rand(gen, R) * 150000).to(torch.int32)
    s["target"] = torch.where(have, s["draft"][(start[s["req"]] + child).clamp(max=R - 1)], other)
    # cached tokens, and pages from one pool: those of the step's tokens are the first of the free ones' former owners
    ctx = (_rand(gen, Q) * 4000).long()
    s["ctx"] = ctx.to(torch.int32)
    held = (ctx + n + PAGE - 1) // PAGE
    if c["op"] == "accept":
        first = held.cumsum(0) - held
        P = Q * 64 + 64
        width = 64
        j = torch.arange(width, device=DEV)[None]
        perm = torch.randperm(P, device=DEV, generator=gen).to(torch.int32)
        s["page_table"] = torch.where(j < held[:, None], perm[(first[:, None] + j).clamp(max=P - 1)], -1).to(torch.int32)
        s["P"] = P
        s["free"] = torch.full((P,), -1, dtype=torch.int32, device=DEV)
        s["free"][:64] = perm[-64:]
        s["free_count"] = _i32([64])
        return s
    # each request's step lies on two pages of its own
    P = 2 * Q + 1
    page = torch.randperm(P, device=DEV, generator=gen)
    at = (ctx % PAGE)[s["req"]] + t
    s["slot"] = (page[2 * s["req"] + at // PAGE] * PAGE + at % PAGE).to(torch.int32)
    s["keys"], s["keys_scale"] = _cache(c, P, gen)
    s["values"], s["values_scale"] = _cache(c, P, gen)
    got = _accepted(s)
    s["accept_len"], s["path"] = got["accept_len"], got["path"]
    return s


def _plan(s):
    import sparse_attention_indexer_launch_gb300 as lib
    c = s["case"]
    if c["op"] in ("prepare", "commit") and c["kv"] != "none":
        s["cache"] = lib.make_kv_cache(s["keys"], s["values"], s["keys_scale"], s["values_scale"])
    if c["op"] == "prepare":
        kind = dict(none=lib.IDX_NORM_NONE, rms=lib.IDX_NORM_RMS, layer=lib.IDX_NORM_LAYER)
        cached = dict(cache=s["cache"], slot=s["slot"]) if c["kv"] != "none" else {}
        s["plan"] = lib.make_norm_rope(
            s["q"], s["k"], s["v"] if c["kv"] in ("bf16", "e4m3") else None, q_out=s["q_out"], k_out=s["k_out"], pos=s["pos"],
            inv_freq=s["inv_freq"], axis=s["axis"], interleaved=c["pairs"] == "interleaved", q_norm=kind[c["norm"]], k_norm=kind[c["k_norm"]],
            q_weight=s["q_weight"], q_bias=s["q_bias"], k_weight=s["k_weight"], k_bias=s["k_bias"], eps=EPS, **cached)
    if c["op"] == "sample":
        s["token"] = torch.empty(c["R"], dtype=torch.int32, device=DEV)
        s["logprob"] = torch.empty(c["R"], dtype=torch.float32, device=DEV)
        s["plan"] = lib.make_sample(s["logits"], s["u"], s["token"], logprob=s["logprob"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if c["op"] == "accept":
        o = s["o"] = dict(new_ctx=torch.empty_like(s["ctx"]), accept_len=torch.empty_like(s["ctx"]), last=torch.empty_like(s["ctx"]),
                          path=torch.empty_like(s["draft"]), token=torch.empty_like(s["draft"]), free_left=torch.empty_like(s["free_count"]))
        s["plan"] = lib.make_tree_accept(s["row_start"], s["draft"], s["target"], s["ctx"], s["page_table"], s["free"], s["free_count"], parent=s["parent"], P=s["P"], **o)
        s["ws"] = lib.alloc_state(lib.tree_accept_state_size())


# ---------------------------------------------------------------------------- run
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_launch_gb300 as lib
    op = s["case"]["op"]
    if op == "prepare":
        lib.idx_norm_rope(s["plan"])
        return _prepared(s)
    if op == "sample":
        lib.idx_sample(s["plan"])
        return dict(token=s["token"], logprob=s["logprob"])
    if op == "accept":
        lib.idx_tree_accept(s["plan"], s["ws"])
        return dict(s["o"], free=s["free"])
    lib.idx_tree_commit(s["cache"], s["row_start"], s["accept_len"], s["path"], s["slot"])
    return _cached(s)


def _run_plain(s):
    return dict(prepare=_plain_prepare, sample=_plain_sample, accept=_plain_accept, commit=_plain_commit)[s["case"]["op"]](s)


def _cached(s):
    return dict(keys=s["keys"], values=s["values"], keys_scale=s["keys_scale"], values_scale=s["values_scale"])


def _prepared(s):
    return dict(q=s["q_out"], k=s["k_out"]) if s["case"]["kv"] == "none" else dict(_cached(s), q=s["q_out"])


def _normed(x, kind, weight, bias):
    x = x.float()
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight + bias
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _rotated(x, cos, sin, rot, pairs):
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_prepare(s):
    c = s["case"]
    angle = s["pos"].t()[:, s["axis_of"]].double() * s["inv_freq"].double()       # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["q_out"].copy_(_rotated(_normed(s["q"], c["norm"], s["q_weight"], s["q_bias"]), cos, sin, c["rot"], c["pairs"]))
    k = _rotated(_normed(s["k"], c["k_norm"], s["k_weight"], s["k_bias"]), cos, sin, c["rot"], c["pairs"])
    if c["kv"] == "none":
        s["k_out"].copy_(k)
        return _prepared(s)
    page, off = s["slot"].long() // PAGE, s["slot"].long() % PAGE
    if c["kv"] == "bf16":
        s["keys"][page, off], s["values"][page, off] = k.bfloat16(), s["v"]
    else:
        code, sc = _quantised(k)
        s["keys"].view(torch.uint8)[page, off], s["keys_scale"][page, :, off] = code.view(torch.uint8), sc
    if c["kv"] == "e4m3":
        code, sc = _quantised(s["v"])
        s["values"].view(torch.uint8)[page, off], s["values_scale"][page, :, off] = code.view(torch.uint8), sc
    return _prepared(s)


def _plain_sample(s):
    """Long sums and values next to a border: 64 bits."""
    x = s["logits"].float()
    R, V = x.shape
    x = torch.where(torch.isnan(x), float("-inf"), x)
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    top = value[:, :1].double()
    rank = torch.arange(V, device=DEV)[None]
    hot = torch.ones(R, 1, dtype=torch.float64, device=DEV) if s["temperature"] is None else s["temperature"].double()[:, None]
    w = torch.exp((value.double() - top) / torch.where(hot > 0, hot, 1.0))
    w = torch.where(hot > 0, w, (rank == 0).double())
    w = torch.where(value == float("-inf"), 0.0, w)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        w = torch.where((rank < k) | (k <= 0), w, 0.0)
    keep = w > 0
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = w.cumsum(1) - w
        keep &= (before < p * w.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None].clamp(max=1)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    upto = w.cumsum(1)
    total = upto[:, -1:]
    i = torch.searchsorted(upto, s["u"].double()[:, None] * total, right=True).clamp(max=V - 1)
    empty = total[:, 0] == 0
    token = torch.where(empty, -1, i[:, 0]).to(torch.int32)
    logprob = torch.where(empty, float("-inf"), torch.log(w.gather(1, i) / total)[:, 0])
    return dict(token=token, logprob=logprob.float())


def _accepted(s):
    """Accepted tokens per request and their numbers, by doubling: after six steps every path of at most 64 nodes is closed."""
    R, req, t = s["R"], s["req"], s["t"]
    first = s["row_start"].long()[req]
    up = torch.where(t > 0, first + (t - 1 if s["parent"] is None else s["parent"].long()), torch.arange(R, device=DEV))
    same = (t > 0) & (s["draft"] == s["target"][up])
    # of several children with the sampled token the first
    lowest = torch.full((R,), R, device=DEV).scatter_reduce_(0, up, torch.where(same, torch.arange(R, device=DEV), R), "amin")
    ok = (t == 0) | (same & (lowest[up] == torch.arange(R, device=DEV)))
    depth = (t > 0).long()
    for _ in range(6):
        ok, depth, up = ok & ok[up], depth + depth[up], up[up]
    accept_len = torch.zeros(s["row_start"].numel() - 1, dtype=torch.long, device=DEV).index_add_(0, req, ok.long())
    # row i of a request's path is its accepted node of depth i: the others are written to a place behind the end
    path = torch.full((R + 1,), -1, dtype=torch.long, device=DEV)
    path[torch.where(ok, first + depth, R)] = t
    return dict(accept_len=accept_len.to(torch.int32), path=path[:R].to(torch.int32))


def _plain_accept(s):
    got = _accepted(s)
    first = s["row_start"].long()[s["req"]]
    path, length, ctx = got["path"].long(), got["accept_len"].long(), s["ctx"].long()
    got["token"] = torch.where(path >= 0, s["target"][first + path.clamp(min=0)], -1).to(torch.int32)
    start = s["row_start"].long()
    n = start[1:] - start[:-1]
    got["last"] = torch.where(length > 0, got["token"][(start[:-1] + length - 1).clamp(0, s["R"] - 1)], -1).to(torch.int32)
    got["new_ctx"] = (ctx + length).to(torch.int32)
    # pages that hold none of the tokens left, in order of requests and positions, onto the stack
    keep, had = (ctx + length + PAGE - 1) // PAGE, (ctx + n + PAGE - 1) // PAGE
    j = torch.arange(s["page_table"].shape[1], device=DEV)[None]
    gone = (j >= keep[:, None]) & (j < had[:, None])
    place = gone.flatten().long().cumsum(0) - 1 + s["free_count"].long()
    place = torch.where(gone.flatten(), place, s["free"].numel())
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[place] = s["page_table"].flatten()
    s["free"].copy_(free[:-1])
    got["free"] = s["free"]
    got["free_left"] = (s["free_count"] + gone.sum()).to(torch.int32)
    return got


def _plain_commit(s):
    first = s["row_start"].long()[s["req"]]
    path, slot = s["path"].long(), s["slot"].long()
    # rows that stay where they are are written over themselves
    to = slot
    at = torch.where(path >= 0, slot[first + path.clamp(min=0)], slot)
    for name in ("keys", "values"):
        x = s[name] if s["case"]["kv"] == "bf16" else s[name].view(torch.uint8)
        x[to // PAGE, to % PAGE] = x[at // PAGE, at % PAGE]
        if s[name + "_scale"] is not None:
            sc = s[name + "_scale"]
            sc[to // PAGE, :, to % PAGE] = sc[at // PAGE, :, at % PAGE]
    return _cached(s)


# ---------------------------------------------------------------------------- 64 bits
def _e4m3_exact(x):
    """Nearest E4M3 value (ties to even) of float64 x with |x| <= 448."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(c, seed):
    return dict(prepare=_exact_prepare, sample=_exact_sample, accept=lambda c, seed: None, commit=_exact_commit)[c["op"]](c, seed)


def _exact_head(x, kind, weight, bias, turn, c):
    """One head of all rows: complex numbers carry the rotated pairs."""
    x = x.double()
    if kind == "layer":
        x = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, unbiased=False, keepdim=True) + EPS) * weight.double() + bias.double()
    elif kind == "rms":
        x = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * weight.double()
    rot, h = c["rot"], c["rot"] // 2
    ia = torch.arange(h, device=DEV) if c["pairs"] == "halves" else 2 * torch.arange(h, device=DEV)
    ib = ia + h if c["pairs"] == "halves" else ia + 1
    z = torch.complex(x[:, ia], x[:, ib]) * turn
    y = x.clone()
    y[:, ia], y[:, ib] = z.real, z.imag
    return y


def _exact_prepare(c, seed):
    s = prepare(c, seed)
    angle = torch.stack([s["pos"][a].double() * f.double() for a, f in zip(s["axis"], s["inv_freq"])], 1)
    turn = torch.polar(torch.ones_like(angle), angle)
    got = {"q": torch.stack([_exact_head(s["q"][:, h], c["norm"], s["q_weight"], s["q_bias"], turn, c) for h in range(c["Hq"])], 1)}
    k = torch.stack([_exact_head(s["k"][:, h], c["k_norm"], s["k_weight"], s["k_bias"], turn, c) for h in range(c["Hkv"])], 1)
    if c["kv"] == "none":
        return dict(got, k=k)
    page, off = s["slot"].long() // PAGE, s["slot"].long() % PAGE
    for name, x in (("keys", k), ("values", s["v"].double())):
        got[name], got[name + "_scale"] = None, None
        if s[name] is None:
            continue
        full = s[name].double()
        if c["kv"] == "bf16":
            full[page, off] = x
        else:
            amax = x.abs().amax(-1)
            sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
            full[page, off] = _e4m3_exact(x / sc[..., None])
            scale = s[name + "_scale"].double()
            scale[page, :, off] = sc
            got[name + "_scale"] = scale
        got[name] = full
    return got


def _exact_sample(c, seed):
    s = prepare(c, seed)
    token, logprob = [], []
    for r in range(c["R"]):
        x = s["logits"][r].double()
        T = 1.0 if s["temperature"] is None else float(s["temperature"][r])
        if T == 0:
            token.append(int((x == x.max()).nonzero()[0]))
            logprob.append(0.0)
            continue
        w = torch.exp((x - x.max()) / T)
        order = torch.argsort(-x, stable=True)
        if s["top_k"] is not None and int(s["top_k"][r]) > 0:
            order = order[:int(s["top_k"][r])]
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            run_ = torch.cumsum(w[order], 0)
            order = order[:1 + int((run_ < float(s["top_p"][r]) * run_[-1]).sum())]
        if s["min_p"] is not None:
            order = order[w[order] >= float(s["min_p"][r])]
        kept = torch.sort(order).values
        run_ = torch.cumsum(w[kept], 0)
        j = int((run_ <= float(s["u"][r]) * float(run_[-1])).sum())
        token.append(int(kept[j]))
        logprob.append(float((x[kept[j]] - x.max()) / T - torch.log(run_[-1])))
    return dict(token=_i32(token), logprob=torch.tensor(logprob, dtype=torch.float64, device=DEV))


def _exact_commit(c, seed):
    s = prepare(c, seed)
    start, length, path = s["row_start"].tolist(), s["accept_len"].tolist(), s["path"].tolist()
    pairs = [(start[i] + path[start[i] + a], start[i] + a) for i in range(c["Q"]) for a in range(length[i])]
    at, to = s["slot"].long()[torch.tensor([p for p, _ in pairs], device=DEV)], s["slot"].long()[torch.tensor([p for _, p in pairs], device=DEV)]
    got = {}
    for name in ("keys", "values"):
        old = s[name].double()
        new = old.clone()
        new[to // PAGE, to % PAGE] = old[at // PAGE, at % PAGE]
        got[name], got[name + "_scale"] = new, None
        if s[name + "_scale"] is not None:
            old = s[name + "_scale"].double()
            new = old.clone()
            new[to // PAGE, :, to % PAGE] = old[at // PAGE, :, at % PAGE]
            got[name + "_scale"] = new
    return got
