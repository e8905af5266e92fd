"""Host-side checks of the step metadata, the 8-bit KV store and the paged attention: the layout
query and the refusals (these calls return before any launch, so no GPU is needed)."""
import ctypes as C

import pytest

from sparse_attention_indexer_mqa_gb300 import binding as Bn


@pytest.fixture(scope="module")
def lib():
    return Bn.load()


@pytest.mark.parametrize("H,D,P", [(1, 64, 64), (8, 128, 128), (3, 128, 64)])
def test_kv_layout(H, D, P):
    lay = Bn.idx_kv_layout(H, D, P)
    assert lay.head_bytes == 2 * P * D + 16 and lay.page_bytes == H * lay.head_bytes
    assert lay.scale_offset == 2 * P * D and lay.scale_block == 16
    assert (lay.kv_heads, lay.head_dim, lay.page_size) == (H, D, P)
    assert lay.head_bytes % 16 == 0


def test_kv_layout_refusals(lib):
    out = Bn.IdxKvLayout()
    assert lib.idx_kv_layout(1, 96, 64, C.byref(out)) == -2
    assert lib.idx_kv_layout(1, 64, 32, C.byref(out)) == -2
    assert lib.idx_kv_layout(0, 64, 64, C.byref(out)) == -1
    assert lib.idx_kv_layout(1, 64, 64, None) == -1


def _meta(lib, **kw):
    d = dict(ctx=16, q=32, B=1, pt=64, w=2, P=64, mk=128, fp=128, fc=4, fs=256, np=8, cu=512, sl=1024,
             pos=2048, sm=4096, T=4, nx=8192)
    d.update(kw)
    return lib.idx_step_meta(d["ctx"], d["q"], d["B"], d["pt"], d["w"], d["P"], d["mk"], d["fp"], d["fc"], d["fs"],
                             d["np"], d["cu"], d["sl"], d["pos"], d["sm"], d["T"], d["nx"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(P=32), -2), (dict(B=16385), -2), (dict(T=1 << 31), -2), (dict(mk=129), -1), (dict(B=-1), -1),
    (dict(T=-1), -1), (dict(ctx=None), -1), (dict(q=None), -1), (dict(cu=None), -1), (dict(pos=None), -1),
    (dict(sm=None), -1), (dict(fs=None), -1), (dict(nx=None), -1), (dict(fp=None), -1), (dict(sl=16), -1),
    (dict(nx=256), -1), (dict(pos=1024), -1), (dict(sm=4100), -1), (dict(ctx=18), -1), (dict(pt=None), -1),
])
def test_step_meta_refusals(lib, kw, want):
    assert _meta(lib, **kw) == want


def _store(lib, **kw):
    d = dict(k=16, v=16, ft=0, n=1, H=1, D=64, kr=64, kh=64, vr=64, vh=64, sm=16, pool=16, np=1, P=64, ps=8208)
    d.update(kw)
    return lib.idx_kv_store(*[d[x] for x in ("k", "v", "ft", "n", "H", "D", "kr", "kh", "vr", "vh", "sm", "pool",
                                             "np", "P", "ps")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ft=2), -1), (dict(n=-1), -1), (dict(H=0), -1), (dict(D=96), -2), (dict(P=16), -2), (dict(ps=8192), -1),
    (dict(ps=8209), -1), (dict(pool=8), -1), (dict(pool=None), -1), (dict(k=None), -1), (dict(v=24), -1),
    (dict(kr=65), -1), (dict(vh=4), -1), (dict(kr=-64), -1), (dict(sm=None), -1), (dict(sm=20), -1),
    (dict(H=2), -1), (dict(H=1025, ps=1 << 30), -2), (dict(n=1 << 31), -2), (dict(n=0, k=None), 0),
])
def test_kv_store_refusals(lib, kw, want):
    assert _store(lib, **kw) == want


def _attn(lib, **kw):
    d = dict(q=16, ft=0, T=1, Hq=4, H=1, D=64, qr=256, qh=64, pool=16, np=1, P=64, ps=8208, pt=16, w=1, sl=16, cu=16,
             B=1, causal=1, mq=1, mk=64, sel=None, ss=0, ns=0, scale=0.125, out=16, orow=256, oh=64, lse=None,
             ws=None, wsb=0)
    d.update(kw)
    return lib.idx_attn_paged(*[d[x] for x in ("q", "ft", "T", "Hq", "H", "D", "qr", "qh", "pool", "np", "P", "ps",
                                               "pt", "w", "sl", "cu", "B", "causal", "mq", "mk", "sel", "ss", "ns",
                                               "scale", "out", "orow", "oh", "lse", "ws", "wsb")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ft=7), -1), (dict(Hq=3, H=2, ps=1 << 20), -1), (dict(Hq=0), -1), (dict(D=80), -2), (dict(P=96), -2),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(mk=65), -1), (dict(sel=16, ss=4, ns=5), -1), (dict(sel=16, ss=4, ns=0), -1), (dict(sel=18, ss=4, ns=4), -1),
    (dict(ns=4), -1), (dict(ws=128, wsb=1 << 20), -1), (dict(q=None), -1), (dict(q=8), -1), (dict(qr=4), -1),
    (dict(out=None), -1), (dict(oh=32), -1), (dict(T=2, orow=32), -1), (dict(pt=None), -1), (dict(sl=None), -1),
    (dict(cu=None), -1), (dict(T=-1), -1), (dict(B=-1), -1), (dict(T=1 << 31), -2), (dict(ps=16), -1),
    (dict(B=1 << 30, T=1 << 20, mq=1 << 10), -2), (dict(T=1 << 28, Hq=8), -2), (dict(sl=18), -1), (dict(lse=6), -1),
    (dict(mk=(1 << 31) - 65536, w=1 << 25), -2), (dict(sel=16, ss=1 << 31, ns=(1 << 31) - 1), -2), (dict(T=0, q=None), 0), (dict(T=0, q=None, ns=4), 0), (dict(B=0), 0), (dict(mq=0), 0),
])
def test_attn_refusals(lib, kw, want):
    assert _attn(lib, **kw) == want


def test_workspace_refusals(lib):
    n = C.c_size_t(0)
    assert lib.idx_attn_workspace_bytes(1, 3, 2, 64, 1, 1, 64, 0, C.byref(n)) == -1
    assert lib.idx_attn_workspace_bytes(1, 2, 2, 65, 1, 1, 64, 0, C.byref(n)) == -2
    assert lib.idx_attn_workspace_bytes(1, 2, 2, 64, 1, 1, 64, 0, None) == -1


def test_binding_refuses_wrong_tensors():
    import torch
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)
    with pytest.raises(ValueError, match="float"):
        Bn.idx_kv_store(z(1, 1, 64, dt=torch.float32), z(1, 1, 64, dt=torch.float32), z(1, dt=torch.int64), None, 0, 64,
                        8208)
    with pytest.raises(ValueError, match="device"):
        Bn.idx_kv_store(z(1, 1, 64, dt=torch.float16), z(1, 1, 64, dt=torch.float16), z(1, dt=torch.int64), None, 0, 64,
                        8208)
    with pytest.raises(ValueError, match="dimensions"):
        Bn.idx_attn_paged(z(1, 64, dt=torch.bfloat16), None, 0, 64, 8208, 1, z(1, 1), z(1), z(2), 0, 1, 64, 1.0,
                          z(1, 64, dt=torch.bfloat16))
