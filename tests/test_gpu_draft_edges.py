"""The drafting step's operators on the GPU where their inputs are unusual: verification with entries that are no probabilities,
or large ones, anywhere in rows of any alignment; page copies with passed-over pairs."""
import math
import subprocess
import sys

import pytest

import draft_ref as dr
from conftest import ROOT
from test_gpu_attn import Bn, torch  # noqa: F401  (fixtures)
from test_gpu_draft import Tree, check_verify, run_verify, walk_inputs

pytestmark = pytest.mark.gpu

NONE = (-0.25, math.nan, math.inf, -math.inf, -2.0 ** -14)  # count as 0 and are reported
UNUSUAL = (-0.0, 2.5, 2.0, 100.0)                           # are what they are


def plant_entries(w, values, places):
    """In every row of sequence b the value b stands for, at the places; never in the tokens that its nodes name."""
    for b, (t0, t1) in enumerate(zip(w["cu"], w["cu"][1:])):
        named = set(w["tokens"][t0:t1])
        at = [x for x in places if x not in named]
        for x in (w["target"], w["draft"]):
            if x is not None:
                x[t0:t1, at] = values[b % len(values)]


def aligned_elsewhere(torch, x, shift):
    """x with rows of an odd distance that begin `shift` elements behind a 16-byte boundary."""
    T, V = x.shape
    wide = torch.full((T, V + (V + 1) % 2), 0.5, dtype=x.dtype, device="cuda")
    flat = torch.full((wide.numel() + 16,), 0.5, dtype=x.dtype, device="cuda")
    y = flat[shift:shift + wide.numel()].view(wide.shape)[:, :V]
    y.copy_(x.cuda())
    return y


@pytest.mark.parametrize("V", [4099, 50001, 131073])
@pytest.mark.parametrize("dt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("drafter", [False, True])
@pytest.mark.parametrize("values,bad", [(NONE, True), (UNUSUAL, False)])
def test_verify_unusual_entries(torch, Bn, V, dt, drafter, values, bad):
    """Odd row lengths, three nodes to a sequence: rows of every alignment. Coins near 1 reject."""
    w = walk_inputs(torch, [3] * 10, V, getattr(torch, dt), 2, V, drafter)
    clean = {k: None if w[k] is None else w[k].clone() for k in ("target", "draft")}
    w["coins"] = [0.99 if t % 2 else 0.6 for t in range(30)]
    for places in ([20], [V // 2, V // 2 + 41], [V - 3, V - 1000], [0, V - 1], [5, V // 3, V // 5 * 4]):
        w.update({k: None if x is None else x.clone() for k, x in clean.items()})
        plant_entries(w, values, places)
        check_verify(torch, Bn, w, 3, Bn.IDX_STATUS_BAD_VALUE if bad else 0)


@pytest.mark.parametrize("dt,shifts", [("float32", range(4)), ("bfloat16", (0, 1, 5, 7))])
@pytest.mark.parametrize("drafter", [False, True])
def test_verify_one_bad_entry(torch, Bn, dt, shifts, drafter):
    """One sequence, one entry: it is reported wherever it lies, and the sums count every other entry once. The drafter's
    rows are aligned like the target's, and unlike them."""
    V = 4099
    for shift in shifts:
        for other in (shift, shift + 1):
            for at in (0, 3, 20, 130, 517, 1024, 2050, 4000, 4098):
                w = walk_inputs(torch, [2], V, getattr(torch, dt), 1, at, drafter)
                w["coins"] = [1.0, 1.0]  # a rejection wherever q > p
                w["target"][:, at] = math.nan
                w["target"] = aligned_elsewhere(torch, w["target"], shift)
                if drafter:
                    w["draft"] = aligned_elsewhere(torch, w["draft"], other)
                for last in (0.9, 0.1):
                    w["last"] = [last]
                    check_verify(torch, Bn, w, 2, Bn.IDX_STATUS_BAD_VALUE)


@pytest.mark.parametrize("B,V,dt", [(100, 70001, "float32"), (200, 70001, "bfloat16"), (310, 1 << 20, "float32"), (310, (1 << 20) - 1, "float16")])
def test_verify_many_requests_reject_without_drafter(torch, Bn, B, V, dt):
    """Four, two and one CTA to a request, whose slice's rejected tokens are marked, up to the whole largest vocabulary. One row
    of probabilities for all nodes."""
    g = torch.Generator().manual_seed(B)
    p = (torch.randn(1, V, generator=g) * 3).softmax(-1).to(getattr(torch, dt))
    heavy = p[0].float().topk(40).indices.tolist()
    tokens = []
    for b in range(B):  # heavy ones, which the draw shows if they stay, and the ends
        pick = torch.randperm(40, generator=g)[:3].tolist()
        tokens += [0, heavy[pick[0]], heavy[pick[1]], heavy[pick[2]], (0, V - 1, V // 2)[b % 3]]
    T = 5 * B
    w = dict(target=p.expand(T, V), draft=None, tokens=tokens, parents=[-1, 0, 0, 0, 0] * B, coins=[0.9999] * T,
             last=torch.rand(B, generator=g).tolist(), cu=[5 * b for b in range(B + 1)])
    dev = dict(w, target=p.cuda().expand(T, V))
    f32 = lambda x: torch.tensor(x, dtype=torch.float32).tolist()  # noqa: E731
    want = dr.verify(w["target"], None, tokens, w["parents"], f32(w["coins"]), f32(w["last"]), w["cu"], 3)
    assert min(want[3]) > 2.0 ** -40
    assert list(run_verify(torch, Bn, dev, 3)) == list(want[:3])


@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
@pytest.mark.parametrize("V", [7, 4098, 4099])
def test_verify_outputs_right_behind_16_bit_rows(torch, Bn, dt, V):
    """Probabilities that begin and end inside a 4-byte word, and a result that begins with the next byte."""
    w = walk_inputs(torch, [1], V, getattr(torch, dt), 1, V, False)
    i32 = dict(dtype=torch.int32, device="cuda")
    memory = torch.zeros(V + 64, dtype=getattr(torch, dt), device="cuda")
    first = V % 2                          # ends on a whole word
    row = memory[first:first + V].view(1, V)
    row.copy_(w["target"].cuda())
    path = memory[first + V:first + V + 4].view(torch.int32).view(1, 2)
    assert path.data_ptr() == row.data_ptr() + 2 * V
    n_path, out, st = torch.zeros(1, **i32), torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
    args = [torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, device="cuda"), torch.tensor(w["last"], dtype=torch.float32, device="cuda"),
            torch.tensor([0, 1], **i32), 1]
    Bn.idx_draft_verify(row, None, *args, path, n_path, out, dev_status=st)
    want = check_verify(torch, Bn, w, 2)
    assert [path.tolist(), n_path.tolist(), out.tolist()] == list(want) and int(st) == 0
    path = memory[first + V - 2:first + V + 2].view(torch.int32).view(1, 2)  # from the row's last word on
    with pytest.raises(Bn.IdxError):
        Bn.idx_draft_verify(row, None, *args, path, n_path, out)


# ------------------------------------------------------------------------------ small trees

@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 1), (64, 16, 2)])
@pytest.mark.parametrize("listed", [False, True])
def test_small_trees_near_one_length_are_cut_alike(torch, Bn, D, Hq, Hkv, listed):
    """No length of a step is an exception among its neighbours: whole below 768 keys, in parts from there on."""
    def wanted(keys):
        n = 8
        return Bn.idx_attn_tree_workspace_bytes(n, Hq, Hkv, D, 1, n, 5000 if listed else keys, keys - n if listed else 0)
    sizes = [256, 384, 511, 512, 513, 520, 600, 640, 766, 767]
    assert [wanted(k) for k in sizes] == [0] * len(sizes)
    assert min(wanted(k) for k in (768, 769, 1024, 1536)) > 0


@pytest.mark.parametrize("keys", [513, 640, 767, 768, 900])
@pytest.mark.parametrize("D,Hq,Hkv,k", [(128, 8, 1, 0), (64, 16, 2, 0), (128, 8, 1, 1), (64, 8, 1, 1)])
def test_small_trees_of_several_steps(torch, Bn, keys, D, Hq, Hkv, k):
    a = Tree(torch, [keys + 300 if k else keys, 70], [8, 3], Hq, Hkv, D, 64, torch.bfloat16, seed=keys)
    sel = a.lists(keys - 8, keys).cuda() if k else None
    a.call(Bn, sel, a.workspace(Bn, keys - 8 if k else 0))
    a.check(sel)


# ------------------------------------------------------------------------------ page copies

@pytest.mark.parametrize("n,layers,page,every", [(64, 16, 8 * 32784, 3), (65, 2, 4352, 1), (7, 1, 16, 2), (1, 3, 8208, 0)])
@pytest.mark.parametrize("seed", range(4))
def test_pages_copy_with_passed_over_pairs(torch, Bn, n, layers, page, every, seed):
    """Pairs that are passed over leave every page alone, the pool's first and last too, which other pairs write or
    read: equal to copies made one pair after the other."""
    g = torch.Generator().manual_seed(seed)
    pages = 2 * n + 3
    others = (torch.randperm(pages - 2, generator=g) + 1)[:2 * n].tolist()
    pairs = [[others[2 * i], others[2 * i + 1]] for i in range(n)]
    pairs[0][seed & 1] = pages - 1              # the last page read, or written
    pairs[-1][1 - (seed & 1)] = 0               # the first page the other way round
    for i in range(n):
        if every and i % (every + 1) == every:
            pairs[i][seed % 2] = -1 - i
    pool = torch.randint(0, 256, (layers, pages, page), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.uint8)
    want = pool.clone()
    for src, dst in pairs:
        if src >= 0 and dst >= 0:
            want[:, dst] = pool[:, src]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Bn.idx_pages_copy(torch.tensor(pairs, dtype=torch.int32, device="cuda"), pool, pages, page, page, layers=layers,
                      layer_stride=pool.stride(0), dev_status=st)
    assert int(st) == 0 and torch.equal(pool, want)


# ------------------------------------------------------------------------------ page rows

FIRST_CALL = r"""
import torch
from sparse_attention_indexer_mqa_gb300 import binding as Bn
i32 = dict(dtype=torch.int32, device="cuda")
pages, B, width = 120000, 200, 100  # enough for a wide cluster
table = torch.arange(B * width, **i32).view(B, width)
lens, parent = torch.full((B,), 64 * width, **i32), torch.arange(B, **i32)
keep = torch.full((B,), 64 * width // 2, **i32)
shares, span = torch.zeros(pages, **i32), torch.tensor([0, pages - B * width], **i32)
free = torch.arange(B * width, pages, **i32)
new_table, new_lens, new_free = torch.full((B, width), -9, **i32), torch.zeros(B, **i32), torch.full((pages,), -9, **i32)
new_span, copies, st = torch.zeros(2, **i32), torch.zeros(B, 2, **i32), torch.zeros(1, **i32)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    Bn.idx_pages_update(parent, keep, table, lens, 64, new_table, new_lens, shares, shares, free, span, new_free, new_span, copies,
                        dev_status=st)
for _ in range(2):
    new_free.fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    half = width // 2
    assert int(st) == 0 and bool((new_table[:, :half] == table[:, :half]).all()) and bool((new_table[:, half:] == -9).all())
    assert new_lens.tolist() == keep.tolist() and not bool(shares.any()) and bool((copies == -1).all())
    back = table[:, half:].reshape(-1)
    assert new_span.tolist() == [0, pages - B * half]
    assert torch.equal(new_free[:pages - B * half], torch.cat([free, back]))
print("fine")
"""


def test_first_wide_update_of_a_process_is_captured(torch):
    """What the device has room for is asked inside the capture."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["fine"], r.stderr[-2000:]
