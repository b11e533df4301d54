"""Arguments that the entry points at the verify step's two ends reject on the host, before any GPU call."""
import ctypes

import pytest
import torch

FAKE = 1 << 20     # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def _cache(lib, **kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, P=8, page_stride=64 * 2 * 128, token_stride=2 * 128, head_stride=128,
             Hkv=2, D=128, kv_dtype=lib.IDX_KV_BF16)
    a.update(kw)
    return lib.KvCache(**a)


def _norm_rope(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=2048, k_stride=2048, v_stride=2048, q_out=2 * FAKE, k_out=None, q_out_stride=512,
             k_out_stride=256, q_weight=FAKE, q_bias=None, k_weight=FAKE, k_bias=None, pos=FAKE, pos_stride=8, inv_freq=FAKE,
             slot=FAKE, rows=None, R=8, Hq=4, Hkv=2, D=128, rot=128, interleaved=0, q_norm=1, k_norm=1, eps=1e-6, axes=1)
    axis = kw.pop("axis", [])
    a.update(kw)
    t = lib.NormRope(**a)
    for i, v in enumerate(axis):
        t.axis[i] = v
    return t


def _call(lib, t, c):
    return lib.lib.idx_norm_rope(None if t is None else ctypes.byref(t), None if c is None else ctypes.byref(c), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=FAKE + 8), dict(q_out=None), dict(k=None), dict(v=None), dict(q_stride=511), dict(q_stride=516),
    dict(k_stride=128), dict(v_stride=128), dict(q_out_stride=256), dict(k_out=FAKE + 2), dict(k_out=3 * FAKE, k_out_stride=8),
    dict(q_out=FAKE), dict(k_out=FAKE), dict(q_weight=FAKE + 4), dict(q_bias=FAKE), dict(q_norm=0), dict(k_norm=3),
    dict(q_norm=-1), dict(pos=None), dict(pos=FAKE + 2), dict(pos_stride=-1), dict(axes=2, pos_stride=7), dict(axes=0),
    dict(axes=5), dict(axis=[0, 1]), dict(inv_freq=None), dict(slot=None), dict(slot=FAKE + 1), dict(rows=FAKE + 2),
    dict(R=-1), dict(Hq=-1), dict(Hq=0), dict(Hkv=0), dict(Hkv=1), dict(D=64), dict(rot=-16), dict(rot=144), dict(eps=0.0),
    dict(eps=2.0), dict(eps=float("nan"))])
def test_norm_rope(lib, kw):
    assert _call(lib, _norm_rope(lib, **kw), _cache(lib)) == lib.IDX_EINVAL


def test_norm_rope_without_a_cache(lib):
    for kw in (dict(), dict(slot=None), dict(slot=None, k_out=2 * FAKE), dict(slot=None, k_out=None, v=None),
               dict(slot=FAKE, k_out=2 * FAKE, v=None), dict(slot=None, v=None, Hkv=0, k_out=2 * FAKE),
               dict(slot=None, v=None, k=None, Hkv=0, Hq=0, q=None, q_out=None)):
        assert _call(lib, _norm_rope(lib, **kw), None) == lib.IDX_EINVAL, kw
    assert _call(lib, None, None) == lib.IDX_EINVAL
    assert _call(lib, _norm_rope(lib, R=0), _cache(lib)) == lib.IDX_OK


def test_norm_rope_limits(lib):
    for kw in (dict(D=96), dict(rot=8), dict(rot=24), dict(Hq=1025), dict(R=2 ** 31 // 8), dict(q_stride=1 << 39),
               dict(pos_stride=1 << 40)):
        kw = dict(dict(slot=None, k_out=2 * FAKE, v=None), **kw)
        assert _call(lib, _norm_rope(lib, **kw), None) == lib.IDX_EUNSUPPORTED, kw
    for kw in (dict(P=2 ** 31 // 64 + 1), dict(D=96)):
        assert _call(lib, _norm_rope(lib), _cache(lib, **kw)) == lib.IDX_EUNSUPPORTED, kw


def test_norm_rope_caches(lib):
    for kw in (dict(k=None), dict(P=0), dict(head_stride=4), dict(kv_dtype=7), dict(k_scale=FAKE), dict(kv_dtype=0),
               dict(kv_dtype=0, k_scale=FAKE), dict(kv_dtype=0, k_scale=FAKE, v_scale=FAKE + 4),
               dict(kv_dtype=0, k_scale=FAKE, v_scale=FAKE, v=None)):
        assert _call(lib, _norm_rope(lib), _cache(lib, **kw)) == lib.IDX_EINVAL, kw
    # keys alone: no values to take
    assert _call(lib, _norm_rope(lib), _cache(lib, v=None)) == lib.IDX_EINVAL


def test_a_cache_without_values_is_for_the_calls_that_say_so(lib):
    c = _cache(lib, v=None)
    assert lib.lib.idx_write_kv(ctypes.byref(c), FAKE, FAKE, 256, FAKE, 4, None) == lib.IDX_EINVAL


def test_norm_rope_binding(lib):
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, inv = torch.zeros(3, dtype=torch.int32), torch.zeros(32)
    good = dict(q_out=q, k_out=k, pos=pos, inv_freq=inv)
    bad = [dict(pos=pos.long()), dict(pos=pos[:2]), dict(inv_freq=inv.double()), dict(axis=[0] * 31), dict(axis=[1] * 32),
           dict(q_weight=torch.ones(32)), dict(q_weight=torch.ones(64).double()), dict(q_out=q[:2]), dict(k_out=q),
           dict(slot=pos[:2]), dict(rows=inv), dict(inv_freq=torch.zeros(129))]
    for kw in bad:
        with pytest.raises(ValueError):
            lib.make_norm_rope(q, k, **dict(good, **kw))
    for args in ((q.float(), k), (q, k[:2]), (q[:, :, ::2], k), (None, None), (q.transpose(0, 1), k)):
        with pytest.raises(ValueError):
            lib.make_norm_rope(*args, **good)
    with pytest.raises(ValueError, match="one GPU"):      # all of it on the CPU
        lib.make_norm_rope(q, k, **good)


def _sample(lib, token=2 * FAKE, logprob=None, **kw):
    a = dict(logits=FAKE, u=FAKE, temperature=FAKE, top_k=FAKE, top_p=FAKE, min_p=FAKE, rows=FAKE, ld=1000, R=4, V=1000,
             logits_dtype=lib.IDX_LOGITS_F32)
    a.update(kw)
    return lib.lib.idx_sample(ctypes.byref(lib.Sample(**a)), token, logprob, None)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(u=None), dict(token=None), dict(logits=FAKE + 2), dict(u=FAKE + 2),
                                dict(logits=FAKE + 1, logits_dtype=1), dict(temperature=FAKE + 1), dict(top_k=FAKE + 1),
                                dict(top_p=FAKE + 2), dict(min_p=FAKE + 3), dict(rows=FAKE + 2), dict(token=FAKE + 2),
                                dict(logprob=FAKE + 2), dict(ld=999), dict(R=0), dict(R=-1), dict(V=0), dict(logits_dtype=2)])
def test_sample(lib, kw):
    assert _sample(lib, **kw) == lib.IDX_EINVAL


def test_sample_limits(lib):
    for kw in (dict(R=65536), dict(V=lib.IDX_MAX_VOCAB + 1, ld=1 << 20), dict(ld=1 << 39)):
        assert _sample(lib, **kw) == lib.IDX_EUNSUPPORTED, kw
    assert lib.lib.idx_sample(None, FAKE, None, None) == lib.IDX_EINVAL


def test_sample_binding(lib):
    x, u, token = torch.zeros(3, 10), torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    for args, kw in (((x.double(), u, token), {}), ((x[0], u, token), {}), ((x.t(), u, token), {}), ((x, u.double(), token), {}),
                     ((x, u[:2], token), {}), ((x, u, token.long()), {}), ((x, u, token[:2]), {}), ((x, u, token), dict(top_k=u)),
                     ((x, u, token), dict(top_p=token)), ((x, u, token), dict(temperature=u[:1])), ((x, u, token), dict(logprob=token)),
                     ((x, u, token), dict(rows=u))):
        with pytest.raises(ValueError):
            lib.make_sample(*args, **kw)
    with pytest.raises(ValueError, match="one GPU"):
        lib.make_sample(x, u, token)


OUTS = ("free_left", "new_ctx", "accept_len", "last", "path", "token")


def _accept(lib, state=FAKE, size=1024, **kw):
    a = {f: FAKE for f in ("row_start", "parent", "draft", "target", "ctx_len", "page_table", "free_pages", "free_count")}
    a.update({n: (2 + i) * FAKE for i, n in enumerate(OUTS)}, P=8, Q=2, pt_stride=4, cap=8, free_cap=8)
    a.update(kw)
    return lib.lib.idx_tree_accept(ctypes.byref(lib.TreeAccept(**a)), state, size, None)


def test_tree_accept(lib):
    for n in ("row_start", "draft", "target", "ctx_len", "page_table", "free_pages", "free_count") + OUTS:
        assert _accept(lib, **{n: None}) == lib.IDX_EINVAL, n
        assert _accept(lib, **{n: FAKE + 2}) == lib.IDX_EINVAL, n
    for kw in (dict(parent=FAKE + 1), dict(Q=0), dict(P=0), dict(pt_stride=0), dict(cap=0), dict(free_cap=-1), dict(path=FAKE),
               dict(token=FAKE), dict(path=FAKE * 9, token=FAKE * 9), dict(state=None), dict(state=FAKE + 512),
               dict(size=lib.tree_accept_state_size() - 1)):
        assert _accept(lib, **kw) == lib.IDX_EINVAL, kw
    for kw in (dict(Q=4097), dict(P=2 ** 31 // 64 + 1), dict(cap=2 ** 31 - 3)):
        assert _accept(lib, **kw) == lib.IDX_EUNSUPPORTED, kw
    assert lib.lib.idx_tree_accept(None, FAKE, 1024, None) == lib.IDX_EINVAL


def test_tree_commit(lib):
    def call(c=None, starts=FAKE, length=FAKE, path=FAKE, slot=FAKE, Q=2, cap=8):
        return lib.lib.idx_tree_commit(ctypes.byref(c or _cache(lib)), starts, length, path, slot, Q, cap, None)

    for kw in (dict(starts=None), dict(length=None), dict(path=None), dict(slot=None), dict(starts=FAKE + 2), dict(length=FAKE + 1),
               dict(path=FAKE + 3), dict(slot=FAKE + 2), dict(Q=0), dict(cap=0), dict(c=_cache(lib, k=None)),
               dict(c=_cache(lib, kv_dtype=0)), dict(c=_cache(lib, head_stride=4)), dict(c=_cache(lib, v=None, v_scale=FAKE))):
        assert call(**kw) == lib.IDX_EINVAL, kw
    for kw in (dict(Q=4097), dict(cap=2 ** 31 - 3), dict(c=_cache(lib, D=256))):
        assert call(**kw) == lib.IDX_EUNSUPPORTED, kw
    assert lib.lib.idx_tree_commit(None, FAKE, FAKE, FAKE, FAKE, 2, 8, None) == lib.IDX_EINVAL


def test_tree_accept_and_commit_binding(lib):
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    good = dict(row_start=i(3), draft=i(8), target=i(8), ctx_len=i(2), page_table=i(2, 4), free_pages=i(6), free_count=i(1), P=8,
                new_ctx=i(2), accept_len=i(2), last=i(2), path=i(8), token=i(8), free_left=i(1))
    for kw in (dict(row_start=i(2)), dict(target=i(7)), dict(page_table=i(3, 4)), dict(page_table=i(8)), dict(path=i(7)),
               dict(token=torch.zeros(8)), dict(last=i(1)), dict(parent=i(7)), dict(free_count=i(0)), dict(draft=i(16)[::2])):
        with pytest.raises(ValueError):
            lib.make_tree_accept(**dict(good, **kw))
    with pytest.raises(ValueError, match="one GPU"):
        lib.make_tree_accept(**good)
    c = _cache(lib)
    for args in ((i(2), i(2), i(8), i(8)), (i(3), i(2), i(8), i(7)), (i(3), i(2).long(), i(8), i(8)), (i(3), i(2), i(16)[::2], i(8))):
        with pytest.raises(ValueError):
            lib.idx_tree_commit(c, *args)
