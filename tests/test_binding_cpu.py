"""What the binding hands to the library, with a library that only records its calls (no GPU)."""
import pytest
import torch

from sparse_attention_indexer_mqa_gb300 import binding as Bn


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors taken for tensors of the current device, and the arguments of each call of the library."""
    made = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                made.append((name, args))
                return 0
            return call

    Bn.load()
    Bn._load_torch()
    monkeypatch.setattr(Bn, "_lib", Library())
    monkeypatch.setattr(Bn, "_device", lambda: -1)
    return made


def attend(T=2, H=4, Hkv=1, D=64, P=64, pages=3, pool=None, stride=None, **kw):
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)
    q = z(T, H, D, dt=torch.float16)
    pool = z(pages, Hkv * (2 * P * D + 16), dt=torch.uint8) if pool is None else pool
    Bn.idx_attn_paged(q, pool, pages, P, pool.stride(0) if stride is None else stride, Hkv, z(T, 2), z(T), z(T + 1), 0,
                      1, 2 * P, 0.125, torch.zeros_like(q), stream=0, **kw)


SEL = 20, 21, 22  # sel_idx, sel_stride, n_sel among the library's arguments


@pytest.mark.parametrize("make", [lambda: torch.zeros(2, 0, dtype=torch.int32),
                                  lambda: torch.zeros(2, 8, dtype=torch.int32)[:, :0],
                                  lambda: torch.zeros(2, 8, dtype=torch.int32)[:, 8:]])
def test_list_without_columns_is_refused(calls, make):
    """A tensor without elements has a null pointer, which would read as no list: every visible key."""
    with pytest.raises(ValueError, match="sel_idx"):
        attend(sel_idx=make())
    assert not calls


def test_lists_reach_the_library(calls):
    sel = torch.zeros(2, 9, dtype=torch.int32)
    attend(sel_idx=sel[:, :7])
    attend()
    attend(T=0, sel_idx=sel[:0, :7])
    attend(T=0, sel_idx=sel[:0, :0])
    got = [[args[i] for i in SEL] for _, args in calls]
    assert got[0] == [sel.data_ptr(), 9, 7]
    assert got[1] == [None, 0, 0]
    assert got[3][0] in (None, 0)


def store(pool, pages, stride, H=1, D=64, P=64):
    k = torch.zeros(1, H, D, dtype=torch.float16)
    Bn.idx_kv_store(k, k.clone(), torch.zeros(1, dtype=torch.int64), pool, pages, P, stride, stream=0)


PAGE = 2 * 64 * 64 + 16


@pytest.mark.parametrize("use", [lambda pool, pages, stride: store(pool, pages, stride),
                                 lambda pool, pages, stride: attend(pool=pool, pages=pages, stride=stride)])
def test_pool_is_measured_by_the_memory_behind_it(calls, use):
    """A view of a wider pool holds its pages though its own elements are fewer than the strides span; one
    that repeats its elements does not."""
    wide = torch.zeros(3, PAGE + 64, dtype=torch.uint8)
    use(wide[:, :PAGE], 3, wide.stride(0))
    use(wide[1:, 16:16 + PAGE], 2, wide.stride(0))
    use(wide[0], 1, wide.stride(0))
    use(wide.view(-1)[:2 * wide.stride(0) + PAGE], 3, wide.stride(0))
    assert len(calls) == 4
    bad = [(wide[:, :PAGE], 4, wide.stride(0)), (wide[1:], 3, wide.stride(0)),
           (wide[2, 65:], 1, PAGE), (wide[0, :PAGE].expand(9, PAGE), 9, PAGE)]
    for pool, pages, stride in bad:
        with pytest.raises(ValueError, match="pool"):
            use(pool, pages, stride)
    assert len(calls) == 4


def test_workspace_without_memory_of_its_own_is_refused(calls):
    """A view that repeats or skips elements claims bytes that are not its own."""
    room = torch.zeros(1 << 16, dtype=torch.uint8)
    attend(workspace=room[256:])
    assert calls[0][1][29] == (1 << 16) - 256
    for ws in (room[:1].expand(1 << 20), room[::2]):
        with pytest.raises(ValueError, match="workspace"):
            attend(workspace=ws)
    assert len(calls) == 1
