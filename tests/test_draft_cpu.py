"""Host-side checks of the drafting step's operators: refusals of the library (these calls return before any launch, so no
GPU is needed), what the binding refuses and hands on, and the plain forms that the GPU tests compare with."""
import ctypes as C
import math
import os
import subprocess

import pytest
import torch

import draft_ref as ref
from sparse_attention_indexer_mqa_gb300 import binding as Bn
from test_binding_cpu import PAGE, Elsewhere, calls  # noqa: F401  (fixture)


@pytest.fixture(scope="module")
def lib():
    return Bn.load()


def _tree(lib, **kw):
    d = dict(q=16, ft=0, T=1, Hq=4, H=1, D=64, qr=256, qh=64, pool=16, np=1, P=64, ps=8208, pt=16, w=1, sl=16, cu=16,
             B=1, mask=16, ms=1, mw=1, mq=1, mk=64, sel=None, ss=0, ns=0, scale=0.125, out=16, orow=256, oh=64, lse=None,
             ws=None, wsb=0)
    d.update(kw)
    return lib.idx_attn_tree(*[d[x] for x in ("q", "ft", "T", "Hq", "H", "D", "qr", "qh", "pool", "np", "P", "ps",
                                              "pt", "w", "sl", "cu", "B", "mask", "ms", "mw", "mq", "mk", "sel", "ss", "ns",
                                              "scale", "out", "orow", "oh", "lse", "ws", "wsb")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(mask=None), -1), (dict(mask=20), -1), (dict(ms=0), -1), (dict(mw=0), -1), (dict(mw=-1), -1),
    (dict(T=65, mq=65), -1), (dict(T=65, mq=65, mw=2, ms=1), -1), (dict(T=1025, mq=1025, mw=17, ms=17), -2),
    (dict(T=2000, mq=1024, mw=15, ms=16), -1), (dict(ft=2), -1), (dict(D=80), -2), (dict(P=96), -2), (dict(scale=0.0), -1),
    (dict(mk=65), -1), (dict(sel=16, ss=4, ns=5), -1), (dict(ns=4), -1), (dict(ws=128, wsb=1 << 20), -1), (dict(q=8), -1),
    (dict(out=None), -1), (dict(T=2, orow=32), -1), (dict(T=-1), -1), (dict(ps=16), -1),
    (dict(sel=16, ss=1 << 31, ns=(1 << 31) - 66000), -2), (dict(T=0, q=None, mask=None, mw=0, ms=0), 0), (dict(B=0), 0),
    (dict(mq=0, mask=None, mw=0, ms=0), 0),
])
def test_tree_refusals(lib, kw, want):
    assert _tree(lib, **kw) == want


def test_tree_workspace(lib):
    n = C.c_size_t(0)
    assert lib.idx_attn_tree_workspace_bytes(1, 3, 2, 64, 1, 1, 64, 0, C.byref(n)) == -1
    assert lib.idx_attn_tree_workspace_bytes(1, 2, 2, 65, 1, 1, 64, 0, C.byref(n)) == -2
    assert lib.idx_attn_tree_workspace_bytes(2048, 2, 2, 64, 1, 1025, 64, 0, C.byref(n)) == -2
    assert lib.idx_attn_tree_workspace_bytes(1, 2, 2, 64, 1, 1, 64, 0, None) == -1


def _verify(lib, **kw):
    d = dict(p=1024, q=2048, ty=2, ts=8, ds=8, T=4, V=8, tok=16, par=32, coin=48, last=64, cu=80, B=1, mq=4, mp=4, path=96,
             n=112, out=128)
    d.update(kw)
    return lib.idx_draft_verify(*[d[x] for x in ("p", "q", "ty", "ts", "ds", "T", "V", "tok", "par", "coin", "last", "cu", "B",
                                                 "mq", "mp", "path", "n", "out")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ty=3), -1), (dict(ty=-1), -1), (dict(T=-1), -1), (dict(V=0), -1), (dict(V=(1 << 20) + 1), -2), (dict(mp=0), -1),
    (dict(B=-1), -1), (dict(mq=-1), -1), (dict(T=1 << 31), -2), (dict(ts=-1), -1), (dict(ds=-8), -1), (dict(p=None), -1),
    (dict(p=1026), -1), (dict(q=2050), -1), (dict(tok=None), -1), (dict(par=None), -1), (dict(coin=None), -1),
    (dict(last=None), -1), (dict(cu=None), -1), (dict(path=None), -1), (dict(n=None), -1), (dict(out=None), -1),
    (dict(tok=18), -1), (dict(path=98), -1), (dict(path=112), -1), (dict(out=16), -1), (dict(n=1024), -1),
    (dict(B=0, p=None, path=None), 0),
])
def test_verify_refusals(lib, kw, want):
    assert _verify(lib, **kw) == want


def _kv(lib, **kw):
    d = dict(path=16, mp=4, n=32, sl=48, cu=64, B=1, pt=80, w=2, pool=1024, H=1, D=64, L=1, ls=0, np=4, P=64, ps=8208, nl=96)
    d.update(kw)
    return lib.idx_kv_compact(*[d[x] for x in ("path", "mp", "n", "sl", "cu", "B", "pt", "w", "pool", "H", "D", "L", "ls", "np",
                                               "P", "ps", "nl")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(H=0), -1), (dict(H=1025, ps=1 << 30), -2), (dict(D=96), -2), (dict(P=32), -2), (dict(ps=8192), -1), (dict(ps=8210), -1),
    (dict(pool=None), -1), (dict(pool=1032), -1), (dict(L=-1), -1), (dict(L=65536, ls=1 << 20), -2), (dict(ls=8), -1),
    (dict(L=2, ls=0), -1), (dict(L=2, ls=3 * 8208), -1), (dict(L=2, ls=8208), -1), (dict(L=3, ls=8208, ps=2 * 8208), -1),
    (dict(B=-1), -1), (dict(mp=-1), -1), (dict(path=None), -1), (dict(n=None), -1), (dict(sl=None), -1), (dict(cu=None), -1),
    (dict(pt=None), -1), (dict(path=18), -1), (dict(nl=98), -1), (dict(nl=48), -1), (dict(w=1 << 26), -2),
    (dict(B=0, path=None, n=None), 0), (dict(L=0, pool=None), 0),
])
def test_kv_compact_refusals(lib, kw, want):
    assert _kv(lib, **kw) == want


def _k(lib, **kw):
    d = dict(path=16, mp=4, n=32, sl=48, cu=64, B=1, pt=80, w=2, dt=0, pool=1024, L=1, ls=0, np=4, P=64, ps=4352, nl=96)
    d.update(kw)
    return lib.idx_k_compact(*[d[x] for x in ("path", "mp", "n", "sl", "cu", "B", "pt", "w", "dt", "pool", "L", "ls", "np", "P",
                                              "ps", "nl")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), -1), (dict(P=16), -2), (dict(ps=4336), -1), (dict(dt=1), -1), (dict(pool=1028), -1), (dict(n=None), -1),
    (dict(L=2, ls=4352), -1), (dict(nl=80), -1), (dict(B=0), 0), (dict(L=0), 0),
])
def test_k_compact_refusals(lib, kw, want):
    assert _k(lib, **kw) == want


def _pages(lib, **kw):
    d = dict(par=16, keep=32, no=2, pt=48, w=2, lens=64, B=2, P=64, nt=80, nw=2, nl=96, sh=112, ns=128, np=8, fp=144, fc=8,
             fs=160, nf=176, nfc=8, nsp=192, cp=208)
    d.update(kw)
    return lib.idx_pages_update(*[d[x] for x in ("par", "keep", "no", "pt", "w", "lens", "B", "P", "nt", "nw", "nl", "sh", "ns",
                                                 "np", "fp", "fc", "fs", "nf", "nfc", "nsp", "cp")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(no=-1), -1), (dict(B=-1), -1), (dict(P=32), -2), (dict(no=16385), -2), (dict(B=16385), -2),
    (dict(np=(1 << 30) + 1, nfc=(1 << 30) + 1), -2), (dict(nfc=7), -1), (dict(par=None), -1), (dict(keep=None), -1),
    (dict(pt=None), -1), (dict(lens=None), -1), (dict(nt=None), -1), (dict(nl=None), -1), (dict(sh=None), -1), (dict(ns=None), -1),
    (dict(fp=None), -1), (dict(fs=None), -1), (dict(nf=None), -1), (dict(nsp=None), -1), (dict(cp=None), -1), (dict(par=18), -1),
    (dict(cp=210), -1), (dict(nt=48), -1), (dict(nl=64), -1), (dict(nf=144), -1), (dict(ns=48), -1), (dict(ns=176), -1),
    (dict(nsp=160), -1), (dict(cp=112), -1),
])
def test_pages_update_refusals(lib, kw, want):
    assert _pages(lib, **kw) == want


def _copy(lib, **kw):
    d = dict(cp=16, n=1, pool=1024, L=1, ls=0, np=4, pb=160, ps=160)
    d.update(kw)
    return lib.idx_pages_copy(*[d[x] for x in ("cp", "n", "pool", "L", "ls", "np", "pb", "ps")], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), -1), (dict(n=65536), -2), (dict(L=65536, ls=1 << 20), -2), (dict(pb=152), -1), (dict(ps=144), -1),
    (dict(ps=168), -1), (dict(cp=None), -1), (dict(cp=18), -1), (dict(pool=None), -1), (dict(pool=1032), -1),
    (dict(L=2, ls=160), -1), (dict(L=2, ls=648), -1), (dict(pb=-16), -1), (dict(pb=0), 0), (dict(n=0, cp=None), 0), (dict(L=0), 0),
])
def test_pages_copy_refusals(lib, kw, want):
    assert _copy(lib, **kw) == want


# ------------------------------------------------------------------------------ binding

z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)  # noqa: E731


def tree(T=2, H=4, D=64, P=64, mask=None, **kw):
    q = z(T, H, D, dt=torch.float16)
    Bn.idx_attn_tree(q, z(3, PAGE, dt=torch.uint8), 3, P, PAGE, 1, z(T, 2), z(T), z(T + 1),
                     z(T, 1, dt=torch.int64) if mask is None else mask, 1, 2 * P, 0.125, torch.zeros_like(q), stream=0, **kw)


def test_masks_reach_the_library(calls):
    wide = z(2, 5, dt=torch.int64)
    tree(mask=wide[:, 1:4])
    tree(mask=wide[:, :1], sel_idx=z(2, 7))
    name, args = calls[0]
    assert name == "idx_attn_tree" and args[17:20] == (wide.data_ptr() + 8, 5, 3) and args[22:25] == (None, 0, 0)
    assert calls[1][1][18:20] == (5, 1) and calls[1][1][24] == 7
    for bad in (z(2, 1), z(3, 1, dt=torch.int64), z(2, dt=torch.int64), z(2, 6, dt=torch.int64)[:, ::2],
                z(1, 2, dt=torch.int64).expand(2, 2)):
        with pytest.raises(ValueError, match="tree_mask"):
            tree(mask=bad)
    assert len(calls) == 2


def verify(T=3, V=5, B=1, target=None, draft=None, **kw):
    d = dict(tokens=z(T), parents=z(T), coins=z(T, dt=torch.float32), last_coins=z(B, dt=torch.float32), cu_seqlens_q=z(B + 1),
             path=z(B, 4), n_path=z(B), out_tokens=z(B, 4))
    d.update(kw)
    Bn.idx_draft_verify(z(T, V, dt=torch.float32) if target is None else target, draft, d["tokens"], d["parents"], d["coins"],
                        d["last_coins"], d["cu_seqlens_q"], 3, d["path"], d["n_path"], d["out_tokens"], stream=0)


def test_probabilities_reach_the_library(calls):
    wide = z(3, 11, dt=torch.bfloat16)
    verify(target=wide[:, 2:7], draft=wide[:, 6:])
    verify(target=z(1, 5, dt=torch.float16).expand(3, 5))
    name, args = calls[0]
    assert name == "idx_draft_verify"
    assert args[:7] == (wide.data_ptr() + 4, wide.data_ptr() + 12, Bn.IDX_BF16, 11, 11, 3, 5)
    assert calls[1][1][1] is None and calls[1][1][2:7] == (Bn.IDX_FP16, 0, 0, 3, 5)
    f = torch.float32
    for kw in (dict(target=z(3, 5, dt=torch.float64)), dict(target=z(3, 10, dt=f)[:, ::2]), dict(target=z(2, 5, dt=f)),
               dict(draft=z(3, 5, dt=torch.float16)), dict(draft=z(3, 4, dt=f)), dict(tokens=z(3, dt=torch.int64)),
               dict(parents=z(2)), dict(coins=z(3, dt=torch.float64)), dict(last_coins=z(2, dt=f)), dict(path=z(2, 4)),
               dict(out_tokens=z(1, 3)), dict(n_path=z(2)), dict(path=z(1, 8)[:, ::2])):
        with pytest.raises(ValueError, match="idx_draft_verify"):
            verify(**kw)
    assert len(calls) == 2


def compact(pool, pages, stride, layers=1, layer_stride=0, **kw):
    d = dict(path=z(1, 3), n_path=z(1), lens=z(1), cu=z(2), table=z(1, 2), new=z(1))
    d.update(kw)
    Bn.idx_kv_compact(d["path"], d["n_path"], d["lens"], d["cu"], d["table"], pool, pages, 64, stride, 1, 64, layers=layers,
                      layer_stride=layer_stride, new_lens=d["new"], stream=0)
    Bn.idx_k_compact(d["path"], d["n_path"], d["lens"], d["cu"], d["table"], Bn.IDX_MXFP4, pool, pages, 64, stride, layers=layers,
                     layer_stride=layer_stride, new_lens=d["new"], stream=0)


def test_layers_have_to_lie_in_the_pool(calls):
    pool = z(2, 3, PAGE, dt=torch.uint8)
    compact(pool, 3, PAGE, 2, 3 * PAGE)
    compact(pool.view(3, 2, PAGE), 3, 2 * PAGE, 2, PAGE)
    compact(pool[1], 3, PAGE)
    Bn.idx_pages_copy(z(4, 2), pool, 3, PAGE, PAGE, layers=2, layer_stride=3 * PAGE, stream=0)
    assert [c[0] for c in calls] == ["idx_kv_compact", "idx_k_compact"] * 3 + ["idx_pages_copy"]
    for bad in ((pool, 3, PAGE, 3, 3 * PAGE), (pool[1], 4, PAGE), (pool[1], 3, PAGE, 2, 3 * PAGE), (pool[1, 2].expand(6, PAGE), 6, PAGE)):
        with pytest.raises(ValueError, match="pool"):
            compact(*bad)
    with pytest.raises(ValueError, match="pool"):
        Bn.idx_pages_copy(z(4, 2), pool, 3, PAGE, PAGE, layers=2, layer_stride=3 * PAGE + 16, stream=0)
    for kw in (dict(path=z(2, 3)), dict(n_path=z(1, dt=torch.int64)), dict(lens=z(2)), dict(cu=z(1)), dict(table=z(2, 2)),
               dict(new=z(2)), dict(path=z(1, 6)[:, ::2]), dict(table=z(2))):
        with pytest.raises(ValueError, match="idx_kv_compact"):
            compact(pool[1], 3, PAGE, **kw)
    with pytest.raises(ValueError, match="copies"):
        Bn.idx_pages_copy(z(4, 3), pool, 3, PAGE, PAGE, stream=0)
    assert len(calls) == 7


def pages(**kw):
    d = dict(parent=z(3), keep=z(3), table=z(2, 4), lens=z(2), new_table=z(3, 4), new_lens=z(3), shares=z(9), new_shares=z(9),
             free=z(9), span=z(2), new_free=z(9), new_span=z(2), copies=z(3, 2))
    d.update(kw)
    Bn.idx_pages_update(d["parent"], d["keep"], d["table"], d["lens"], 64, d["new_table"], d["new_lens"], d["shares"],
                        d["new_shares"], d["free"], d["span"], d["new_free"], d["new_span"], d["copies"], stream=0)


def test_page_rows_reach_the_library(calls):
    pages()
    pages(new_table=z(3, 9), new_free=z(20))
    assert calls[0][1][2] == 3 and calls[0][1][13] == 9 and calls[1][1][9] == 9 and calls[1][1][18] == 20
    for kw in (dict(keep=z(2)), dict(lens=z(3)), dict(new_table=z(2, 4)), dict(new_lens=z(4)), dict(new_shares=z(8)),
               dict(new_free=z(8)), dict(span=z(3)), dict(copies=z(3, 3)), dict(parent=z(3, dt=torch.int64)),
               dict(table=z(2, 8)[:, ::2])):
        with pytest.raises(ValueError, match="idx_pages_update"):
            pages(**kw)
    assert len(calls) == 2


def test_status_word_of_the_drafting_calls(calls):
    pool = z(3, PAGE, dt=torch.uint8)
    lists = z(1, 3), z(1), z(1), z(2), z(1, 2)
    uses = [lambda **kw: tree(**kw),
            lambda **kw: Bn.idx_kv_compact(*lists, pool, 3, 64, PAGE, 1, 64, stream=0, **kw),
            lambda **kw: Bn.idx_k_compact(*lists, 0, pool, 3, 64, PAGE, stream=0, **kw),
            lambda **kw: Bn.idx_pages_copy(z(1, 2), pool, 3, PAGE, PAGE, stream=0, **kw)]
    word = z(1)
    for use in uses:
        use(dev_status=word)
        assert calls[-1][1][-2] == word.data_ptr()
        for bad in (Elsewhere(), z(1, dt=torch.int64), z(0)):
            with pytest.raises(ValueError, match="dev_status"):
                use(dev_status=bad)
    assert len(calls) == len(uses)


# ------------------------------------------------------------------------------ the plain forms themselves

def sampled(p, q, fan, seed, trials):
    """First emitted tokens of `trials` walks over `fan` children drawn from q."""
    g = torch.Generator().manual_seed(seed)
    n = fan + 1
    tokens = torch.multinomial(q.double(), trials * n, replacement=True, generator=g)
    coins, last = torch.rand(trials * n, generator=g), torch.rand(trials, generator=g)
    cu = [n * b for b in range(trials + 1)]
    rows = lambda x: x.expand(trials * n, -1)  # noqa: E731
    _, _, out, _ = ref.verify(rows(p), rows(q), tokens.tolist(), ([-1] + [0] * fan) * trials, coins.tolist(), last.tolist(), cu, 2)
    return torch.bincount(torch.tensor([o[0] for o in out]), minlength=len(p))


@pytest.mark.parametrize("fan", [1, 2, 4])
def test_walk_emits_the_targets_distribution(fan):
    """Chi-square of 20000 first tokens over 6 values, 5 degrees of freedom: above 30 with a chance of 1.5e-5."""
    p = torch.tensor([0.4, 0.05, 0.05, 0.3, 0.2, 0.0])
    q = torch.tensor([0.1, 0.3, 0.2, 0.1, 0.1, 0.2])
    n = sampled(p, q, fan, 1, 20000)
    want = p.double() * 20000
    assert n[5] == 0
    assert float(((n - want) ** 2 / want.clamp(min=1e-9))[:5].sum()) < 30


def test_hand_worked_walk():
    """p = (.5, .25, .25), q = (.25, .75, 0). Child 1 (token 1, coin .5): .5 * .75 >= .25, rejected; c = 1, S = .5.
    Child 2 (token 0, coin .9): .9 * .25 * .5 < .5 - .25, accepted. Behind it a draw at .6 of (.2, .2, .6): token 2."""
    p = torch.tensor([[.5, .25, .25], [1, 0, 0], [.2, .2, .6]])
    q = torch.tensor([[.25, .75, 0], [1, 0, 0], [1, 0, 0]])
    path, n, out, _ = ref.verify(p, q, [9, 1, 0], [-1, 0, 0], [0, .5, .9], [.6], [0, 3], 3)
    assert (path, n, out) == ([[0, 2, -1]], [2], [[0, 2, -1]])
    # both rejected: c = 1.5, S = .125; left of p: (.125, 0, .25)
    path, n, out, near = ref.verify(p, q, [9, 1, 1], [-1, 0, 0], [0, .5, .9], [.34], [0, 3], 3)
    assert (path, n, out) == ([[0, -1, -1]], [1], [[2, -1, -1]])
    assert math.isclose(near[0], .34 - 1 / 3, rel_tol=1e-6)
    # without the drafter's: token 1 goes (S = .75), then token 0: .9 * .75 >= .5; token 2 is left
    path, n, out, _ = ref.verify(p, None, [9, 1, 0], [-1, 0, 0], [0, .5, .9], [.99], [0, 3], 3)
    assert (path, n, out) == ([[0, -1, -1]], [1], [[2, -1, -1]])


def test_hand_worked_pages():
    """Pages of 64: row 0 (100 tokens: pages 5, 6) goes on twice and to 64 tokens, row 1 (70: 7, 8) ends."""
    t, lens, shares, free, span, copies, status = ref.pages_update(
        [0, 0, 0], [100, 100, 64], [[5, 6], [7, 8]], [100, 70], 64, [[-1, -1]] * 3, [0] * 10, [1, 2, 3], [1, 3], [-9] * 10)
    assert t == [[5, 6], [5, 2], [5, -1]] and lens == [100, 100, 64]
    assert shares == [0, 0, 0, 0, 0, 2, 0, 0, 0, 0] and copies == [[-1, -1], [6, 2], [-1, -1]]
    assert free[:3] == [3, 7, 8] and span == [0, 3] and status == 0


# ------------------------------------------------------------------------------ arrays that overlap in part

@pytest.mark.parametrize("kw", [
    dict(path=36), dict(path=28), dict(path=84), dict(n=84), dict(n=104), dict(out=100), dict(out=60, mp=2), dict(out=1148),
    dict(n=2172), dict(path=16384, B=1 << 30, mp=1 << 30, n=1 << 60, out=1 << 61),
])
def test_verify_refuses_partial_overlap(lib, kw):
    """Addresses that are nobody's first one: a word of an output inside an input (path in parents, tokens or lengths, out in coins,
    the last probability of either side), of an output inside another, and sizes whose product passes 64 bits."""
    assert _verify(lib, **kw) == -1


@pytest.mark.parametrize("kw", [dict(nl=20), dict(nl=28), dict(nl=68), dict(nl=84), dict(B=3, n=128, sl=144, cu=160, pt=192, nl=152),
                                dict(B=2, n=128, sl=144, cu=160, pt=192, nl=140)])
def test_compact_refuses_partial_overlap(lib, kw):
    """new_lens inside the path, the row bounds, the table or the lengths, and running into them from in front."""
    assert _kv(lib, **kw) == -1
    assert _k(lib, **kw) == -1


_APART = dict(par=4096, keep=4112, pt=4128, lens=4160, nt=4224, nl=4256, sh=4352, ns=4416, fp=4480, fs=4544, nf=4608, nsp=4672,
              cp=4736)


@pytest.mark.parametrize("kw", [
    dict(nl=4100), dict(nl=4108), dict(nt=4120), dict(nt=4132), dict(cp=4164), dict(nl=4156), dict(ns=4356), dict(ns=4324),
    dict(nf=4484), dict(nsp=4548), dict(nsp=4540), dict(nf=4420), dict(cp=4228), dict(nsp=4740),
])
def test_pages_update_refuses_partial_overlap(lib, kw):
    """A word of an output inside parent, keep, table, lengths, counts (new counts are the counts as a whole or apart from them),
    free pages or their span, and of one output inside another."""
    assert _pages(lib, **{**_APART, **kw}) == -1


# ------------------------------------------------------------------------------ free lists without pages of their own

@pytest.mark.parametrize("kw", [dict(nf=None), dict(nf=None, nfc=1), dict(nf=None, no=0, B=0)])
def test_pages_update_refuses_a_free_list_without_memory(lib, kw):
    """No page is counted, yet what is left of free_pages is passed on to new_free."""
    assert _pages(lib, **{**_APART, "np": 0, "sh": None, "ns": None, **kw}) == -1


def test_pages_update_without_any_list_reaches_the_launch(calls):
    """Empty tensors have null pointers: the binding hands them on with length 0."""
    pages(shares=z(0), new_shares=z(0), free=z(0), new_free=z(0))
    args = calls[0][1]
    assert args[13] == 0 and args[15] == 0 and args[18] == 0


# ------------------------------------------------------------------------------ a device without room for a wide cluster

def test_pages_update_takes_a_narrow_cluster_where_no_wide_one_fits(tmp_path):
    """The choice, compiled for the host with fakes of the device's answer: some room, none, and a query that failed."""
    csrc = os.path.join(os.path.dirname(Bn.__file__), "csrc")
    main = tmp_path / "plan.cpp"
    main.write_text(r"""
#include <stdio.h>
#include "pages_plan.h"
int main() {
    const int64_t entries[] = {0, 1, idx::kMany, idx::kMany + 1, int64_t(1) << 40};
    const int fits[] = {-1, 0, 1, 9};
    for (int64_t n : entries)
        for (int f : fits) {
            int asked = 0;
            const int ctas = idx::pages_ctas(n, [&] { ++asked; return f; });
            printf("%d %d ", ctas, asked);
        }
}
""")
    subprocess.run(["g++", "-std=c++17", "-I" + csrc, str(main), "-o", str(tmp_path / "plan")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "plan")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [8, 0] * 12 + [8, 1, 8, 1, 16, 1, 16, 1] * 2
