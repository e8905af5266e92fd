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
