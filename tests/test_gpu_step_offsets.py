"""The calls around a verify step where offsets pass 31 and 32 bits: what they give there equals,
to the bit, what they give on the same data laid out small."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def spread(shape, stride, dtype=torch.bfloat16):
    """[R][..] with rows `stride` elements apart, uninitialised."""
    inner = int(np.prod(shape[1:]))
    strides = [stride] + [int(np.prod(shape[i + 1:])) for i in range(1, len(shape))]
    return torch.empty((shape[0] - 1) * stride + inner, dtype=dtype, device="cuda").as_strided(shape, strides)


@pytest.mark.parametrize("dtype,stride", [(torch.bfloat16, 2 ** 31 + 8), (torch.float32, 2 ** 30 + 3)])
def test_logits_far_apart(lib, dtype, stride):
    gen = torch.Generator(device="cuda").manual_seed(1)
    R, V = 4, 9001
    x = torch.randn(R, V, device="cuda", generator=gen).to(dtype)
    far = spread((R, V), stride, dtype)
    far.copy_(x)
    u, p = torch.rand(R, device="cuda", generator=gen), torch.full((R,), 0.9, device="cuda")
    got = [(torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")) for _ in range(2)]
    for t, (token, logprob) in zip((x, far), got):
        lib.idx_sample(lib.make_sample(t, u, token, logprob=logprob, top_p=p))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_caches_and_rows_past_32_bits(lib, kv):
    """Norm, rotation and moves at the ends of a cache of 2^32 elements, from rows 2^31 elements apart."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    R, Hq, Hkv, D = 3, 4, 8, 128
    pages = 2 ** 32 // (PAGE * Hkv * D) + 2
    e = torch.bfloat16 if kv == "bf16" else torch.uint8
    x = torch.randn(R, Hq + 2 * Hkv, D, device="cuda", generator=gen).bfloat16()
    far = spread(x.shape, 2 ** 31 + 16)
    far.copy_(x)
    weight = torch.rand(D, device="cuda", generator=gen)
    inv_freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda").float() / D)

    def caches(P):
        k, v = (torch.empty(P, PAGE, Hkv, D, dtype=e, device="cuda") for _ in "kv")
        ks, vs = (torch.empty(P, Hkv, PAGE, device="cuda") if kv == "e4m3" else None for _ in "kv")
        return k, v, ks, vs

    big, small, outs = caches(pages), caches(pages % 5 + 3), []
    last, few = pages * PAGE - 1, small[0].shape[0] * PAGE - 1
    for data, (k, v, ks, vs), end in ((far, big, last), (x, small, few)):
        q = torch.empty(R, Hq, D, dtype=torch.bfloat16, device="cuda")
        cache, slot = lib.make_kv_cache(k, v, ks, vs), i32([end, 5, end - 70])
        lib.idx_norm_rope(lib.make_norm_rope(data[:, :Hq], data[:, Hq:Hq + Hkv], data[:, Hq + Hkv:], q_out=q, pos=i32([2 ** 31 - 1, 7, 123456789]),
                                             inv_freq=inv_freq, cache=cache, slot=slot, q_weight=weight, k_weight=weight))
        # row 2's token to row 1's slot, then row 1's path ends; the same the other way for request 1
        lib.idx_tree_commit(cache, i32([0, 3]), i32([2]), i32([0, 2, -1]), i32([end, 6, end - 70]))
        lib.idx_tree_commit(cache, i32([0, 3]), i32([2]), i32([0, 2, -1]), i32([5, end - 140, end]))
        at = torch.tensor([end, 5, end - 70, 6, end - 140], device="cuda")
        outs.append([q] + [t[at // PAGE, at % PAGE] for t in (k, v)] + [t[at // PAGE, :, at % PAGE] for t in (ks, vs) if t is not None])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    k = outs[0][1]
    assert torch.equal(k[3], k[2]) and torch.equal(k[4], k[0])


def test_page_tables_past_32_bits(lib):
    """Pages given back from rows of a page table that lie 2^32 entries behind its first."""
    Q, stride = 4096, 2 ** 20 + 3
    table = torch.empty(Q, stride, dtype=torch.int32, device="cuda")
    ctx = np.full(Q, 64 * (stride - 2))
    ctx[::2] = 64
    first = torch.tensor(ctx // 64, device="cuda").long()
    rows = torch.arange(Q, device="cuda")
    table[rows, first] = (2 * rows).int()
    table[rows, first + 1] = (2 * rows + 1).int()
    new = 20
    draft, target = np.zeros(Q * new, int), np.ones(Q * new, int)     # token 0 alone
    o = {n: i32(np.full(k, -9)) for n, k in (("new_ctx", Q), ("accept_len", Q), ("last", Q), ("path", Q * new), ("token", Q * new), ("free_left", 1))}
    ctx[1::4] += 50        # (50 + 20 tokens: token 0 in a page, the last in the next)
    stack = i32(np.full(2 * Q, -5))
    state = lib.alloc_state(lib.tree_accept_state_size())
    lib.idx_tree_accept(lib.make_tree_accept(i32(np.arange(Q + 1) * new), i32(draft), i32(target), i32(ctx), table, stack, i32([0]), P=2 * Q, **o), state)
    assert lib.last_device_status(state) == lib.IDX_OK
    assert (o["accept_len"] == 1).all() and (o["new_ctx"].cpu().numpy() == ctx + 1).all()
    want = [2 * i + 1 for i in range(1, Q, 4)]
    assert o["free_left"].item() == len(want) and stack[:len(want)].tolist() == want
