"""The binding of the verify step takes tensors of one GPU only: no address of host memory, or of
another GPU's, reaches a kernel.  No GPU is needed: the tensors stand in for their places."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_indexer_launch_gb300 as lib
    return lib


class On:
    """A tensor that says it is on the GPU of that index; everything else is the tensor's own."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _table_tensors(index):
    a = dict(ctx_len=_i32(2), new_len=_i32(2), page_table=_i32(2, 4), free_pages=_i32(8), free_count=_i32(1), row_start=_i32(3),
             free_left=_i32(1), row_req=_i32(8), row_bound=_i32(8), row_pos=_i32(8), slot=_i32(8),
             mask=torch.zeros(8, dtype=torch.int64), parent=_i32(8))
    return {k: On(v, index) for k, v in a.items()}


def test_tables(lib):
    good = _table_tensors(3)
    assert lib.make_tree_tables(P=8, **good).device == 3
    for name, x in good.items():
        for other in (-1, 2):
            with pytest.raises(ValueError):
                lib.make_tree_tables(P=8, **dict(good, **{name: On(x.t, other)}))


def _cache_tensors(index, f8):
    k, v = (torch.zeros(2, 64, 2, 64, dtype=torch.uint8 if f8 else torch.bfloat16) for _ in "kv")
    a = [k, v] + ([torch.zeros(2, 2, 64), torch.zeros(2, 2, 64)] if f8 else [])
    return [On(x, index) for x in a]


@pytest.mark.parametrize("f8", [False, True])
def test_cache(lib, f8):
    good = _cache_tensors(1, f8)
    assert lib.make_kv_cache(*good).device == 1
    for n, x in enumerate(good):
        for other in (-1, 0):
            with pytest.raises(ValueError):
                lib.make_kv_cache(*good[:n], On(x.t, other), *good[n + 1:])


def _problem_args(lib, index):
    return dict(q=On(torch.zeros(3, 4, 64, dtype=torch.bfloat16), index), cache=lib.make_kv_cache(*_cache_tensors(index, False)),
                page_table=On(_i32(1, 2), index), ctx_len=On(_i32(1), index), row_start=On(_i32(2), index),
                mask=On(torch.zeros(3, dtype=torch.int64), index), max_ctx=64, max_new=3, scale=0.1)


def test_problem(lib):
    good = _problem_args(lib, 1)
    assert lib.make_tree_problem(**good).device == 1
    for name, x in good.items():
        if name == "cache":
            bad = [lib.make_kv_cache(*_cache_tensors(0, False))]
        elif isinstance(x, On):
            bad = [On(x.t, -1), On(x.t, 0)]
        else:
            continue
        for y in bad:
            with pytest.raises(ValueError):
                lib.make_tree_problem(**dict(good, **{name: y}))


def _calls(lib):
    """Each call with its tensors by name, on GPU 1, and a function that makes the call."""
    tables = lib.make_tree_tables(P=8, **_table_tensors(1))
    cache = lib.make_kv_cache(*_cache_tensors(1, False))
    problem = lib.make_tree_problem(**_problem_args(lib, 1))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    attn = dict(out=bf(3, 4, 64), state=torch.zeros(64, dtype=torch.uint8), lse=torch.zeros(3, 4))
    yield tables, dict(state=torch.zeros(1024, dtype=torch.uint8)), lambda **a: lib.idx_tree_tables(tables, **a)
    yield cache, dict(k_new=bf(3, 2, 64), v_new=bf(3, 2, 64), slot=_i32(3)), lambda **a: lib.idx_write_kv(cache, **a)
    yield problem, attn, lambda **a: lib.idx_tree_attention(problem, **a)
    yield problem, dict(attn, sel=_i32(3, 5)), lambda **a: lib.idx_tree_attention_selected(problem, **a)


def test_calls(lib, monkeypatch):
    reached = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(lib, "_check", lambda status, what: reached.append(what))   # (there is no GPU to answer)
    for plan, tensors, call in _calls(lib):
        on = {k: On(v, 1) for k, v in tensors.items()}
        n = len(reached)
        for name, x in on.items():
            for other in (-1, 0):
                with pytest.raises(ValueError):
                    call(**dict(on, **{name: On(x.t, other)}))
        # every tensor on one GPU, which is not the current one
        with monkeypatch.context() as m:
            m.setattr(torch._C, "_cuda_getDevice", lambda: 0)
            with pytest.raises(ValueError):
                call(**on)
        # a plan of another GPU
        plan.device = 0
        with pytest.raises(ValueError):
            call(**on)
        plan.device = 1
        assert len(reached) == n
