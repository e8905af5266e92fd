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


class Elsewhere:
    """An int32 that is not on the current device (a host tensor, as the fixture has it)."""
    dtype, device, shape, nbytes = torch.int32, "elsewhere", (1,), 4
    is_contiguous = lambda self: True
    get_device = lambda self: 3
    numel = dim = lambda self: 1
    stride = lambda self: (1,)
    data_ptr = lambda self: 4096


def meta(**kw):
    z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt)
    Bn.idx_step_meta(z(1), z(1), z(2).view(1, 2), 64, 128, z(4), z(2), 8, z(2), z(1), z(3), z(3, torch.int64), z(1), stream=0,
                     **kw)


def store_one(**kw):
    k = torch.zeros(1, 1, 64, dtype=torch.float16)
    Bn.idx_kv_store(k, k.clone(), torch.zeros(1, dtype=torch.int64), torch.zeros(PAGE, dtype=torch.uint8), 1, 64, PAGE,
                    stream=0, **kw)


@pytest.mark.parametrize("use", [meta, store_one, attend])
def test_status_word_has_to_be_on_the_device(calls, use):
    """The kernels write to it: a pointer that is not the device's would fault there."""
    word = torch.zeros(1, dtype=torch.int32)
    for status in (word, word.data_ptr(), None):
        use(dev_status=status)
    assert [args[-2] for _, args in calls] == [word.data_ptr(), word.data_ptr(), None]
    for bad in (Elsewhere(), torch.zeros(1, dtype=torch.int64), torch.zeros(1), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="dev_status"):
            use(dev_status=bad)
    assert len(calls) == 3
