"""Plans and caches carry addresses of tensors: they keep those tensors."""
import gc
import weakref

import pytest
import torch


@pytest.fixture
def lib(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_launch_gb300 as lib
    monkeypatch.setattr(lib, "_one_device", lambda *tensors: 0)     # tensors of the CPU stand for a GPU's
    return lib


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def bf16(*n):
    return torch.zeros(*n, dtype=torch.bfloat16)


def kept(build):
    """build(note) makes a plan of tensors that nothing else refers to; note() is told each."""
    refs = []

    def note(t):
        refs.append(weakref.ref(t))
        return t

    plan = build(note)
    gc.collect()
    alive = [r() is not None for r in refs]
    del plan
    gc.collect()
    return alive, [r() is not None for r in refs]


def cache(lib, note):
    f8 = lambda: note(torch.zeros(2, 64, 1, 128, dtype=torch.uint8))  # noqa: E731
    scale = lambda: note(torch.ones(2, 1, 64))  # noqa: E731
    return lib.make_kv_cache(f8(), f8(), scale(), scale())


def keys_alone(lib, note):
    return lib.make_kv_cache(note(bf16(2, 64, 1, 128)), None)


def norm_rope(lib, note):
    x = lambda *n: note(bf16(*n))  # noqa: E731
    w = lambda: note(torch.ones(128))  # noqa: E731
    return lib.make_norm_rope(x(3, 4, 128), x(3, 1, 128), x(3, 1, 128), q_out=x(3, 4, 128), k_out=x(3, 1, 128), pos=note(i32(3)),
                              inv_freq=note(torch.ones(64)), cache=cache(lib, note), slot=note(i32(3)), q_weight=w(), q_bias=w(),
                              k_weight=w(), k_bias=w(), rows=note(i32(1)))


def sample(lib, note):
    f = lambda: note(torch.ones(3))  # noqa: E731
    return lib.make_sample(note(torch.zeros(3, 10)), f(), note(i32(3)), logprob=f(), temperature=f(), top_k=note(i32(3)), top_p=f(),
                           min_p=f(), rows=note(i32(1)))


def accept(lib, note):
    n = lambda *s: note(i32(*s))  # noqa: E731
    return lib.make_tree_accept(n(3), n(8), n(8), n(2), n(2, 4), n(6), n(1), P=8, new_ctx=n(2), accept_len=n(2), last=n(2), path=n(8),
                                token=n(8), free_left=n(1), parent=n(8))


def tables(lib, note):
    n = lambda *s: note(i32(*s))  # noqa: E731
    return lib.make_tree_tables(n(2), n(2), n(2, 4), n(6), n(1), P=8, row_start=n(3), free_left=n(1), row_req=n(8), row_bound=n(8),
                                row_pos=n(8), slot=n(8), mask=note(torch.zeros(8, dtype=torch.int64)), parent=n(8))


def attention(lib, note):
    return lib.make_tree_problem(note(bf16(8, 4, 128)), cache(lib, note), note(i32(2, 4)), note(i32(2)), note(i32(3)),
                                 note(torch.zeros(8, dtype=torch.int64)), 256, 8, 1.0)


def problem(lib, note):
    return lib.make_problem(note(bf16(3, 64, 128)), note(torch.ones(3, 64)), note(torch.zeros(2, 64, 128, dtype=torch.uint8)),
                            note(torch.ones(2, 64)), note(i32(2, 4)), note(i32(3)), note(i32(3)), 256, lib.IDX_KV_E4M3)


@pytest.mark.parametrize("build", [cache, keys_alone, norm_rope, sample, accept, tables, attention, problem])
def test_tensors_live_as_long_as_the_plan(lib, build):
    alive, after = kept(lambda note: build(lib, note))
    assert all(alive) and not any(after)
