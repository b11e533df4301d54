"""Inputs and 64-bit references of the tree-verify step's tests.

The references follow the formulas in include/idx.h row by row in float64, share
nothing with the library and never look at a masked position's values."""
from __future__ import annotations

import numpy as np
import torch

PAGE = 64


def random_tree(rng, n):
    """Parents of a random tree: token 0 a root, token t under an earlier one."""
    return [-1 if t == 0 else int(rng.integers(0, t)) for t in range(n)]


def ancestor_masks(parents):
    got = []
    for t, p in enumerate(parents):
        got.append((1 << t) | (got[p] if p >= 0 else 0))
    return got


def as_int64(masks):
    return [m - (1 << 64) if m >> 63 else m for m in masks]


class Step:
    """Device tensors of a step: `ctx` cached and `new` drafted tokens per request.

    layout: "token" [P][64][Hkv][D], "head" [P][Hkv][64][D], or "pair" (K and V of a
    page interleaved in one allocation).  Cache slots that no request uses hold NaN."""

    def __init__(self, ctx, new, Hq, Hkv, D, kv="bf16", layout="token", masks=None, seed=0, q_pad=0, extra_pages=2,
                 first_page=0, amp=1.0):
        import sparse_attention_indexer_launch_gb300 as lib
        self.lib, self.ctx, self.new = lib, list(ctx), list(new)
        self.Hq, self.Hkv, self.D, self.kv = Hq, Hkv, D, kv
        Q, R = len(ctx), sum(new)
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        pages = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new)]
        P = first_page + sum(pages) + extra_pages
        self.P = P
        perm = first_page + rng.permutation(sum(pages) + extra_pages)
        table = np.full((Q, max(pages + [1]) + 1), -1, np.int32)
        at = 0
        for i, n in enumerate(pages):
            table[i, :n] = perm[at:at + n]
            at += n
        self.table = table
        self.page_table = torch.from_numpy(table).cuda()
        if layout == "head":
            k, v = (torch.empty(P, Hkv, PAGE, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in "kv")
        elif layout == "pair":
            both = torch.empty(P, 2, PAGE, Hkv, D, dtype=torch.bfloat16, device="cuda")
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = (torch.empty(P, PAGE, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.k_scale = self.v_scale = None
        if kv == "e4m3":
            # codes in the same order of dimensions as the bf16 tensors above
            k, v = (torch.empty_strided(x.shape, x.stride(), dtype=torch.uint8, device="cuda") for x in (k, v)) if layout != "pair" else \
                (lambda b: (b[:, 0], b[:, 1]))(torch.empty(P, 2, PAGE, Hkv, D, dtype=torch.uint8, device="cuda"))
            self.k_scale, self.v_scale = (torch.full((P, Hkv, PAGE), float("nan"), device="cuda") for _ in "kv")
        self.k, self.v = k, v
        for x in (k, v):     # stale slots
            x[first_page:].fill_(0x7F if kv == "e4m3" else float("nan"))
        for i in range(Q):
            j = np.arange(ctx[i] + new[i])
            if not j.size:
                continue
            page = torch.from_numpy(table[i, j // PAGE].astype(np.int64)).cuda()
            off = torch.from_numpy(j % PAGE).cuda()
            for x, sc in ((k, self.k_scale), (v, self.v_scale)):
                val = torch.randn(j.size, Hkv, D, device="cuda", generator=gen) * amp
                if kv == "bf16":
                    x[page, off] = val.bfloat16()
                else:
                    s = val.abs().amax(-1) / 448.0
                    x[page, off] = (val / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                    sc[page, :, off] = s
        wide = torch.empty(R, Hq * D + q_pad, dtype=torch.bfloat16, device="cuda")
        wide.normal_(generator=gen)
        self.q = wide[:, :Hq * D].unflatten(1, (Hq, D))
        self.masks = masks
        self.mask = None if masks is None else torch.tensor(as_int64(masks), dtype=torch.int64, device="cuda")
        self.start = [0]
        for n in new:
            self.start.append(self.start[-1] + n)
        self.row_start = torch.tensor(self.start, dtype=torch.int32, device="cuda")
        self.ctx_len = torch.tensor(list(ctx), dtype=torch.int32, device="cuda")
        self.R, self.scale = R, D ** -0.5
        self.cache = lib.make_kv_cache(self.k, self.v, self.k_scale, self.v_scale)

    def problem(self, **kw):
        p = self.lib.make_tree_problem(self.q, self.cache, self.page_table, self.ctx_len, self.row_start, self.mask,
                                       max(self.ctx + [0]), max(self.new + [1]), self.scale)
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    def attend(self, sel=None, problem=None, state=None, stream=None):
        p = problem if problem is not None else self.problem()
        out = torch.full((self.R, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.R, self.Hq), 7.0, dtype=torch.float32, device="cuda")
        self.state = state if state is not None else self.lib.alloc_state(
            self.lib.tree_state_size(p, 0 if sel is None else sel.shape[1]))
        if sel is None:
            self.lib.idx_tree_attention(p, out, self.state, lse=lse, stream=stream)
        else:
            self.lib.idx_tree_attention_selected(p, sel, out, self.state, lse=lse, stream=stream)
        return out, lse

    def status(self):
        return self.lib.last_device_status(self.state)

    def values(self, i, j, h):
        """K and V of request i's positions j at head h, float64."""
        page = torch.from_numpy(self.table[i, j // PAGE].astype(np.int64)).cuda()
        off = torch.from_numpy(j % PAGE).cuda()
        got = []
        for x, sc in ((self.k, self.k_scale), (self.v, self.v_scale)):
            if self.kv == "bf16":
                got.append(x[page, off, h].double())
            else:
                got.append(x[page, off, h].view(torch.float8_e4m3fn).double() * sc[page, h, off].double()[:, None])
        return got

    def reference(self, sel=None):
        """(out, lse, tolerance of out, tolerance of lse), float64.

        The tolerances follow from the arithmetic that idx.h states.  A score is an
        fp32 sum of D products, off by at most e = 2^-16 scale sum_d |q_d k_d| (D 2^-23
        for a truncating sum of up to 128 terms), so a probability is off by the factor
        exp(+-2e); rounding it to bf16 adds 2^-9 of it, the exponential and the fp32
        sums 2^-18.  The output is rounded to bf16: 2^-9 of it (2^-8 at the bottom of a
        binade counts half a unit of 2^-7)."""
        G = self.Hq // self.Hkv
        out = torch.zeros(self.R, self.Hq, self.D, dtype=torch.float64, device="cuda")
        lse = torch.full((self.R, self.Hq), float("-inf"), dtype=torch.float64, device="cuda")
        tol = torch.full_like(out, 1e-30)
        tol_lse = torch.zeros_like(lse)
        for i in range(len(self.ctx)):
            for t in range(self.new[i]):
                r = self.start[i] + t
                m = (2 << t) - 1 if self.masks is None else self.masks[r]
                seen = np.array([u for u in range(self.new[i]) if (m >> u) & 1], dtype=np.int64) + self.ctx[i]
                if sel is None:
                    cached = np.arange(self.ctx[i], dtype=np.int64)
                else:
                    s = sel[r].cpu().numpy().astype(np.int64)
                    cached = s[(s >= 0) & (s < self.ctx[i])]
                j = np.concatenate([cached, seen])
                if not j.size:
                    continue
                for h in range(self.Hkv):
                    k, v = self.values(i, j, h)
                    q = self.q[r, h * G:(h + 1) * G].double()
                    s = q @ k.T * self.scale
                    z = torch.logsumexp(s, 1)
                    p = torch.exp(s - z[:, None])
                    o = p @ v
                    hs = slice(h * G, (h + 1) * G)
                    out[r, hs], lse[r, hs] = o, z
                    e = 2.0 ** -16 * (q.abs() @ k.abs().T).amax(1) * self.scale
                    tol[r, hs] = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -18 + 2 * e)[:, None] * (p @ v.abs()) + 1e-30
                    tol_lse[r, hs] = e + 2.0 ** -18 + 2.0 ** -22 * z.abs()
        return out, lse, tol, tol_lse


def check(step, out, lse, sel=None):
    ro, rl, to, tl = step.reference(sel)
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty), "rows that see nothing differ"
    assert bool((out[empty] == 0).all()), "a row that sees nothing is not zero"
    assert torch.equal(torch.isfinite(out.double()), torch.isfinite(ro)), "non-finite outputs differ"
    fine = torch.isfinite(ro)
    bad = ((out.double() - ro).abs() > to) & fine
    assert not bool(bad.any()), (f"{int(bad.sum())} values outside tolerance, first at {bad.nonzero()[0].tolist()}: worst "
                                 f"{float(((out.double() - ro).abs() / to)[fine].max()):.3g} of it")
    rest = ~empty & torch.isfinite(rl)
    d = (lse.double() - rl).abs()[rest]
    assert bool((d <= tl[rest]).all()), f"lse off by {float((d / tl[rest]).max()):.3g} of its tolerance"
