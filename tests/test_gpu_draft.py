"""The drafting step's operators on the GPU against the plain forms of tests/draft_ref.py: whole numbers and bytes
equal, attention within the bounds that attn_ref.attention derives."""
import math

import pytest

import attn_ref as ref
import draft_ref as dr
from test_gpu_attn import Att, Bn, torch  # noqa: F401  (fixtures, inputs)
from test_gpu_attn_edges import plant

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ attention of a tree

class Tree(Att):
    """Att's rows as nodes of random trees; every hole-th node is padding that sees nothing of its tree."""

    def __init__(self, torch, lens, nq, Hq, Hkv, D, P, dt, seed=0, pad=0, fan=4, hole=0, words_extra=0, **kw):
        super().__init__(torch, lens, nq, Hq, Hkv, D, P, dt, seed, pad, **kw)
        g = torch.Generator().manual_seed(seed)
        self.sets = []
        for n in nq:
            self.sets += [set() if hole and j % hole == hole - 1 else s for j, s in enumerate(dr.ancestors(dr.random_tree(n, g, fan)))]
        self.words = -(-max(nq) // 64) + words_extra
        self.mask()

    def mask(self):
        torch = self.torch
        m = dr.mask_words(self.sets + [set()] * (self.T - len(self.sets)), self.words)
        # behind a sequence's nodes anything may stand
        for b, n in enumerate(self.nq):
            for j in range(n, 64 * self.words):
                bit = 1 << j % 64
                m[self.cu[b]:self.cu[b + 1], j // 64] |= bit - (1 << 64) if bit >> 63 else bit
        self.tree = m.cuda()

    def call(self, Bn, sel=None, ws=None, **kw):
        args = dict(lse=self.lse, sel_idx=sel, workspace=ws, dev_status=self.status)
        args.update(kw)
        Bn.idx_attn_tree(self.q, self.pool, self.pages, self.P, self.pool.stride(0), self.Hkv, self.table, self.dev_lens,
                         self.dev_cu, self.tree, max(self.nq), max(self.lens), self.scale, self.out, **args)

    def workspace(self, Bn, n_sel=0):
        n = Bn.idx_attn_tree_workspace_bytes(self.T, self.Hq, self.Hkv, self.D, len(self.lens), max(self.nq), max(self.lens), n_sel)
        return self.torch.full((max(n, 256),), 255, dtype=self.torch.uint8, device="cuda")

    def keys(self, sel=None):
        return dr.keys_of(self.sets, self.nq, self.lens, self.T, sel).cuda()

    def check(self, sel=None, status=0):
        super().check(0, self.keys(sel), status)

    def lists(self, k, seed):
        """Lists of k entries: keys in front of the tree, and entries that do not count (a node's position too)."""
        torch = self.torch
        g = torch.Generator().manual_seed(seed)
        sel = torch.full((self.T, k), -1, dtype=torch.int32)
        for b, n in enumerate(self.lens):
            front = n - self.nq[b]
            for t in range(self.cu[b], self.cu[b + 1]):
                ids = torch.randperm(max(front, 0), generator=g)[:max(0, k - 5)]
                row = torch.cat([ids, torch.tensor([-1, front, n - 1, 2147483647, -2147483648])])
                row = row[torch.randperm(len(row), generator=g)][:k]
                sel[t, :len(row)] = row.int()
        return sel.cuda()


SHAPES = [  # lens, rows, heads: mma.sync rows, tensor-memory tiles, many words of mask, a tree longer than a step
    ([9, 40, 300, 130], [1, 5, 8, 2], 4, 1), ([64, 129, 0, 31], [3, 1, 2, 16], 4, 2), ([500, 17, 1], [16, 16, 1], 2, 1),
    ([40, 300, 77], [8, 20, 31], 16, 2), ([200, 130, 64, 900], [1, 33, 64, 12], 8, 1), ([70, 260], [67, 130], 12, 4),
    ([400, 300], [300, 7], 3, 1), ([30, 5, 16, 0], [30, 5, 16, 4], 8, 2), ([20, 3], [40, 9], 4, 1)]


@pytest.mark.parametrize("lens,nq,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("D,P,dt", [(64, 64, "float16"), (128, 128, "bfloat16"), (128, 64, "float16")])
def test_tree(torch, Bn, lens, nq, Hq, Hkv, D, P, dt):
    a = Tree(torch, lens, nq, Hq, Hkv, D, P, getattr(torch, dt), Hq + D, pad=2, hole=7)
    a.call(Bn, ws=a.workspace(Bn))
    a.check()
    a.out.fill_(77)
    a.lse.fill_(77)
    a.call(Bn)
    a.check()


@pytest.mark.parametrize("lens,nq,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("D,P,dt", [(64, 128, "bfloat16"), (128, 64, "float16")])
@pytest.mark.parametrize("k", [6, 140])
def test_tree_listed(torch, Bn, lens, nq, Hq, Hkv, D, P, dt, k):
    a = Tree(torch, lens, nq, Hq, Hkv, D, P, getattr(torch, dt), Hq + D + k, pad=1, hole=9)
    sel = a.lists(k, k)
    a.call(Bn, sel, a.workspace(Bn, k))
    a.check(sel)


@pytest.mark.parametrize("Hq", [1, 8, 40])
@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 1024])
def test_any_mask(torch, Bn, Hq, n):
    """Masks that are no trees: random bits on either side of the diagonal, rows of none and of all."""
    a = Tree(torch, [n + 37, n], [n, n], Hq, 1, 64, 64, torch.float16, n + Hq, words_extra=1)
    g = torch.Generator().manual_seed(n)
    rows = sorted({0, min(1, n - 1), n // 2, n - 1})
    dense = torch.rand(2 * n, n, generator=g) < 0.3
    dense[0], dense[n - 1] = False, True
    a.sets = [set(x.nonzero()[:, 0].tolist()) for x in dense]
    a.mask()
    a.call(Bn, ws=a.workspace(Bn))
    keep = rows + [n + r for r in rows]
    keys = a.keys()
    # the reference walks row by row: compared on a few
    o, l, otol, ltol = ref.attention(a.q[keep], a.pool, 64, 1, a.table[[0] * len(rows) + [1] * len(rows)],
                                     [a.lens[r // n] for r in keep], list(range(len(keep) + 1)), 0, a.scale, keys[keep])
    assert int(a.status) == 0
    assert ((a.out[keep].double() - o).abs() <= otol).all()
    some = l > -math.inf
    assert (a.lse[keep].double()[~some] == -math.inf).all()
    assert ((a.lse[keep].double() - l).abs()[some] <= ltol[some]).all()


@pytest.mark.parametrize("Hq,Hkv,D,n", [(8, 1, 128, 4), (8, 1, 64, 40), (64, 8, 128, 16), (3, 1, 128, 9)])
def test_lower_triangle_is_causal(torch, Bn, Hq, Hkv, D, n):
    """A chain's mask gives what idx_attn_paged gives, bit for bit: the same kernels, splits and order."""
    a = Tree(torch, [5000, n, 300], [n] * 3, Hq, Hkv, D, 64, torch.bfloat16, n, fan=1)
    ws = a.workspace(Bn)
    a.call(Bn, ws=ws)
    out, lse = a.out.clone(), a.lse.clone()
    Att.call(a, Bn, 1, ws=ws)
    assert torch.equal(out, a.out) and torch.equal(lse, a.lse)


@pytest.mark.parametrize("Hq,Hkv,D,nq", [(4, 1, 128, 6), (64, 1, 128, 3), (16, 2, 64, 33)])
@pytest.mark.parametrize("k", [0, 2048])
def test_tree_split(torch, Bn, Hq, Hkv, D, nq, k):
    """A key axis in several parts, the nodes in the last; same call, same bits; with less workspace; without."""
    a = Tree(torch, [9000, 4100], [nq, nq], Hq, Hkv, D, 64, torch.float16, nq + k)
    sel = a.lists(k, 3) if k else None
    ws = a.workspace(Bn, k)
    assert ws.numel() > 256
    a.call(Bn, sel, ws)
    a.check(sel)
    first, l1 = a.out.clone(), a.lse.clone()
    ws.fill_(0)
    a.call(Bn, sel, ws)
    assert torch.equal(first, a.out) and torch.equal(l1, a.lse)
    a.call(Bn, sel, ws[:ws.numel() // 3 // 256 * 256])
    a.check(sel)
    a.call(Bn, sel)
    a.check(sel)


@pytest.mark.parametrize("D,k,heads", [(128, 300, 64), (64, 1030, 48), (128, 140, 128)])
def test_many_lists_at_once(torch, Bn, D, k, heads):
    """Thousands of units of the tensor-memory kernel, whose lookups and products run side by side on every SM, against 16
    heads at a time, which take the other kernel. Either is within its own bound of the exact result, about 2^-10 of the
    weighted codes; rows of 300 keys add up to less than 64."""
    a = Tree(torch, [5000, 3000], [1000, 900], heads, 1, D, 64, torch.float16, k, fan=1)
    g = torch.Generator(device="cuda").manual_seed(k)
    sel = torch.randint(0, 2000, (a.T, k), generator=g, device="cuda", dtype=torch.int32)
    sel[:, ::7] = torch.randint(-5, 9000, sel[:, ::7].shape, generator=g, device="cuda", dtype=torch.int32)
    a.call(Bn, sel, a.workspace(Bn, k))
    out, lse = a.out.clone(), a.lse.clone()
    a.call(Bn, sel, a.workspace(Bn, k))
    assert torch.equal(out, a.out) and torch.equal(lse, a.lse)
    q = a.q
    for h in range(0, heads, 16):
        a.q, a.Hq = q[:, h:h + 16], 16
        a.out, a.lse = torch.zeros_like(a.q), torch.zeros(a.T, 16, device="cuda")
        a.call(Bn, sel)
        assert int(a.status) == 0
        assert float((a.lse - lse[:, h:h + 16]).abs().max()) < 1e-4
        assert float((a.out.float() - out[:, h:h + 16].float()).abs().max()) < 64 * 2.0 ** -9


@pytest.mark.parametrize("Hq,nq,D", [(4, 6, 128), (8, 40, 64), (64, 5, 128), (2, 140, 128), (2, 9, 64)])
@pytest.mark.parametrize("long", [False, True])
def test_tree_nan_codes(torch, Bn, Hq, nq, D, long):
    """NaN codes among the nodes reach the rows that see them and no others, though those lie in the same tile; the two
    that a row sees need not be the lowest."""
    extra = 5000 if long else 11
    a = Tree(torch, [nq + extra, nq + 70], [nq, nq], Hq, 1, D, 64, torch.bfloat16, nq)
    ws = a.workspace(Bn) if long else None
    a.call(Bn, ws=ws)
    clean, cl = a.out.clone(), a.lse.clone()
    f = [n - nq for n in a.lens]
    marks = [(0, f[0] + 2, 1, 5), (0, f[0] + nq - 1, 1, 8), (0, f[0] + nq // 2, 1, D - 1), (1, f[1] + 1, 0, 7), (1, f[1] + nq - 2, 1, 0)]
    for m in marks:
        plant(a, *m)
    a.call(Bn, ws=ws)
    hit = torch.zeros(a.T, D, dtype=torch.bool, device="cuda")
    seen = torch.zeros(a.T, dtype=torch.bool, device="cuda")
    hit_lse = seen.clone()
    for b, pos, side, dim in marks:
        for t in range(a.cu[b], a.cu[b + 1]):
            if pos - f[b] in a.sets[t]:
                seen[t] = True
                if side:
                    hit[t, dim] = True
                else:
                    hit[t], hit_lse[t] = True, True
    assert int(a.status) == 0 and bool(seen.any()) and not bool(seen.all())
    assert torch.equal(a.out[~seen], clean[~seen]) and torch.equal(a.lse[~hit_lse], cl[~hit_lse])
    assert a.out.transpose(1, 2)[hit].isnan().all() and a.lse[hit_lse].isnan().all()
    left = (seen[:, None] & ~hit)[:, None].expand_as(a.out) & ~a.out.isnan()
    assert torch.equal(a.out[left], clean[left])
    # in front of the tree every row sees it
    a.out.copy_(clean)
    plant(a, 0, 1, 1, 3)
    a.call(Bn, ws=ws)
    assert a.out[:nq, :, 3].isnan().all()


@pytest.mark.parametrize("Hq,nq,k", [(4, 3, 0), (16, 20, 0), (4, 3, 30), (64, 3, 30)])
def test_tree_bad_pages_and_lengths(torch, Bn, Hq, nq, k):
    a = Tree(torch, [200, 100, 150], [nq] * 3, Hq, 1, 128, 64, torch.bfloat16)
    sel = a.lists(k, 1) if k else None
    a.call(Bn, sel)
    a.check(sel)
    before = a.out.clone()
    good = a.table.clone()
    a.table[0, 0] = a.pages
    a.call(Bn, sel)
    assert int(a.status) == Bn.IDX_STATUS_BAD_PAGE and torch.equal(a.out[nq:], before[nq:]) and a.out.isfinite().all()
    a.status.zero_()
    a.table = good
    for lens in ([201, 100, 150], [-1, 100, 150]):
        a.out.fill_(77)
        a.dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        a.call(Bn, sel)
        assert int(a.status) == Bn.IDX_STATUS_BAD_LEN and (a.out[:nq] == 77).all() and torch.equal(a.out[nq:], before[nq:])
        a.status.zero_()
    a.dev_lens = torch.tensor(a.lens, dtype=torch.int32, device="cuda")
    a.dev_cu = torch.tensor([0, nq, 2 * nq, 3 * nq + 5], dtype=torch.int32, device="cuda")
    a.out.fill_(77)
    a.call(Bn, sel)
    assert int(a.status) == Bn.IDX_STATUS_BAD_LEN
    assert torch.equal(a.out[:2 * nq], before[:2 * nq]) and (a.out[2 * nq:] == 77).all()


@pytest.mark.parametrize("Hq,nq", [(4, 3), (8, 30)])
def test_tree_strides_and_non_finite_queries(torch, Bn, Hq, nq):
    """q a slice of a wider projection, out and masks with strides of their own; a NaN in q stays in its row."""
    a = Tree(torch, [150, 40], [nq, nq], Hq, 2, 64, 64, torch.float16, stride_extra=48)
    wide = torch.randn(a.T, 3, Hq, 64, device="cuda").half()
    wide[:, 1] = a.q
    a.q = wide[:, 1]
    big = torch.full((a.T, Hq + 2, 64), 77.0, device="cuda").half()
    a.out = big[:, 1:-1]
    m = torch.full((a.T, a.words + 3), -1, dtype=torch.int64, device="cuda")
    m[:, 1:1 + a.words] = a.tree
    a.tree = m[:, 1:1 + a.words]
    a.call(Bn)
    a.check()
    assert (big[:, 0] == 77).all() and (big[:, -1] == 77).all()
    before = a.out.clone()
    a.q[1, 1, 3] = math.inf
    a.call(Bn)
    assert a.out[1, 1].isnan().all()
    a.out[1, 1] = before[1, 1]
    assert torch.equal(a.out, before)


def test_tree_streams_graphs_and_offsets(torch, Bn):
    """On another stream, captured and replayed with other masks, pages behind 2^32 bytes."""
    a = Tree(torch, [300, 40], [6, 6], 8, 2, 128, 64, torch.bfloat16)
    a.call(Bn)
    want = a.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.out.fill_(77)
    s.wait_stream(torch.cuda.current_stream())
    a.call(Bn, stream=s)
    s.synchronize()
    assert torch.equal(a.out, want)
    ws = a.workspace(Bn)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(Bn, ws=ws)
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        a.sets = sum((dr.ancestors(dr.random_tree(6, gen)) for _ in range(2)), [])
        kept = a.tree
        a.mask()
        kept.copy_(a.tree)
        a.tree = kept
        a.out.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        a.check()
    stride = (1 << 32) // a.pages + (1 << 20)
    big = torch.zeros(a.pages, stride // 16 * 16, dtype=torch.uint8, device="cuda")
    big[:, :a.pool.shape[1]] = a.pool
    a.pool = big
    a.out.fill_(77)
    a.call(Bn)
    a.check()


# ------------------------------------------------------------------------------ verification

def walk_inputs(torch, nq, V, dt, fan, seed, drafter, pad=0):
    g = torch.Generator().manual_seed(seed)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    T = cu[-1] + pad
    target = (torch.randn(T, V, generator=g) * 2).softmax(-1)
    draft = ((target.log() + torch.randn(T, V, generator=g)) * 0.8).softmax(-1)
    parents, tokens = [], []
    for b, n in enumerate(nq):
        p = dr.random_tree(n, g, fan)
        for j in range(n):
            parents.append(p[j])
            tokens.append(int(torch.multinomial(draft[cu[b] + max(p[j], 0)], 1, generator=g)))
    return dict(target=target.to(dt), draft=draft.to(dt) if drafter else None, tokens=tokens + [0] * pad, parents=parents + [0] * pad,
                coins=torch.rand(T, generator=g).tolist(), last=torch.rand(len(nq), generator=g).tolist(), cu=cu)


def run_verify(torch, Bn, w, max_path, status=0, max_q=None, stream=None):
    i32 = dict(dtype=torch.int32, device="cuda")
    B = len(w["cu"]) - 1
    path, n_path, out = torch.full((B, max_path), -7, **i32), torch.full((B,), -7, **i32), torch.full((B, max_path), -7, **i32)
    st = torch.zeros(1, **i32)
    on = lambda x: None if x is None else x.cuda()  # noqa: E731
    f = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    nq = [y - x for x, y in zip(w["cu"], w["cu"][1:])]
    Bn.idx_draft_verify(on(w["target"]), on(w["draft"]), torch.tensor(w["tokens"], **i32), torch.tensor(w["parents"], **i32),
                        f(w["coins"]), f(w["last"]), torch.tensor(w["cu"], **i32), max(nq) if max_q is None else max_q, path, n_path,
                        out, dev_status=st)
    assert int(st) == status
    return path.tolist(), n_path.tolist(), out.tolist()


def check_verify(torch, Bn, w, max_path, status=0):
    got = run_verify(torch, Bn, w, max_path, status)
    # fp32 values in 64 bits on both sides: a border nearer than 2^-40 of the sum would be a coincidence
    f32 = lambda x: torch.tensor(x, dtype=torch.float32).tolist()  # noqa: E731
    want = dr.verify(w["target"], w["draft"], w["tokens"], w["parents"], f32(w["coins"]), f32(w["last"]), w["cu"], max_path)
    assert min(want[3], default=1.0) > 2.0 ** -40
    assert got[0] == want[0]
    assert got[1] == want[1]
    assert got[2] == want[2]
    return got


@pytest.mark.parametrize("V", [1, 2, 31, 33, 257, 1000, 4099, 32768])
@pytest.mark.parametrize("dt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("drafter", [False, True])
def test_verify(torch, Bn, V, dt, drafter):
    w = walk_inputs(torch, [5, 1, 0, 9, 33, 2, 40], V, getattr(torch, dt), 3, V, drafter, pad=2)
    check_verify(torch, Bn, w, 12)
    check_verify(torch, Bn, w, 1)


@pytest.mark.parametrize("V,drafter", [(131072, True), (131071, False), (1 << 20, True), (1 << 20, False)])
def test_verify_large_vocabularies(torch, Bn, V, drafter):
    w = walk_inputs(torch, [4, 7], V, torch.float32, 6, 5, drafter)
    for i, coin in enumerate([0.999, 0.9999, 0.5]):
        w["coins"] = [coin] * len(w["coins"])
        w["last"] = [0.1 + 0.3 * i, 0.9999999]
        check_verify(torch, Bn, w, 4)


@pytest.mark.parametrize("drafter", [False, True])
def test_verify_many_siblings_and_long_chains(torch, Bn, drafter):
    """100 children of one node, all of them rejected in some walks; a chain that is accepted whole; 1000 nodes."""
    w = walk_inputs(torch, [101] * 6 + [60] * 3 + [1000], 50, torch.float32, 1, 9, drafter)
    for b in range(6):
        w["parents"][w["cu"][b] + 1:w["cu"][b + 1]] = [0] * 100
    w["coins"][:300] = [0.99999] * 300
    for t in range(w["cu"][6], w["cu"][9]):
        w["coins"][t] = 0.0
    got = check_verify(torch, Bn, w, 70)
    assert got[1][6:9] == [60] * 3


@pytest.mark.parametrize("drafter", [False, True])
def test_verify_odd_inputs(torch, Bn, drafter):
    """Tokens outside the vocabulary, parents that are not lower, rows without probabilities, entries that are none, coins
    at the ends and outside."""
    w = walk_inputs(torch, [6, 6, 6, 6, 3], 40, torch.float32, 2, 3, drafter)
    w["tokens"][1], w["tokens"][2] = -1, 40
    w["parents"][6 + 3], w["parents"][6 + 4] = 3, 5
    check_verify(torch, Bn, w, 6, Bn.IDX_STATUS_BAD_VALUE)
    w = walk_inputs(torch, [6, 6, 6, 6, 3], 40, torch.float32, 2, 4, drafter)
    w["target"][0] = 0.0           # nothing to accept, nothing to draw
    w["target"][6:12, 5] = math.nan
    w["target"][6:12, 7] = -0.25
    w["target"][6:12, 9] = math.inf
    got = check_verify(torch, Bn, w, 6, Bn.IDX_STATUS_BAD_VALUE)
    assert got[2][0] == [-1] * 6 and got[1][0] == 1
    w = walk_inputs(torch, [1, 1, 1, 1, 1, 1], 40, torch.float32, 2, 5, drafter)
    w["target"][:, 0] = 0.0
    w["target"][:, 39] = 0.0
    w["last"] = [0.0, 1.0 - 2.0 ** -24, 0.5, 0.25, 2.0 ** -30, 0.75]
    got = check_verify(torch, Bn, w, 2)
    assert got[2][0][0] == 1 and got[2][4][0] == 1
    for last, want in ((1.0, 38), (7.0, 38), (math.inf, 38), (-0.5, 1), (math.nan, 1)):
        w["last"] = [last] * 6
        got = run_verify(torch, Bn, w, 2, Bn.IDX_STATUS_BAD_VALUE)
        assert [o[0] for o in got[2]] == [want] * 6


def test_verify_equal_distributions(torch, Bn):
    """p = q: every child is accepted; with c = 1 nothing is left, and the draw falls back on p."""
    w = walk_inputs(torch, [4] * 50, 300, torch.float32, 1, 6, True)
    w["draft"] = w["target"].clone()
    got = check_verify(torch, Bn, w, 4)
    assert got[1] == [4] * 50
    w["coins"] = [math.nan] * len(w["coins"])  # compares false: rejected
    got = check_verify(torch, Bn, w, 4)
    assert got[1] == [1] * 50 and all(0 <= o[0] < 300 for o in got[2])


def test_verify_small_differences(torch, Bn):
    """p and q a few units of the last place apart: what is left after a rejection is rounding-sized and still exact."""
    w = walk_inputs(torch, [5] * 40, 2000, torch.float32, 4, 7, True)
    g = torch.Generator().manual_seed(1)
    bump = 1 + torch.randint(-3, 4, w["target"].shape, generator=g) * 2.0 ** -23
    w["draft"] = (w["target"].double() * bump).float()
    w["coins"] = [math.nan if t % 2 else 0.99 for t in range(len(w["coins"]))]
    check_verify(torch, Bn, w, 3)


@pytest.mark.parametrize("dt,V,extra,shift", [("float32", 1003, 5, 1), ("bfloat16", 1001, 7, 3), ("float16", 999, 1, 1), ("float32", 64, 0, 0)])
def test_verify_strides(torch, Bn, dt, V, extra, shift):
    """Rows at any alignment, other ones for the two sides, and one row for all nodes."""
    dt = getattr(torch, dt)
    w = walk_inputs(torch, [7, 3, 12], V, dt, 3, 2, True)
    plain = check_verify(torch, Bn, w, 8)
    T = w["target"].shape[0]
    wide = torch.full((T, V + extra + 8), 0.5, dtype=dt, device="cuda")
    wide[:, shift:shift + V] = w["target"].cuda()
    other = torch.full((T, V + 2 * extra + 3), 0.5, dtype=dt, device="cuda")
    other[:, 2:2 + V] = w["draft"].cuda()
    v = dict(w, target=wide[:, shift:shift + V], draft=other[:, 2:2 + V]) if extra else w
    assert run_verify(torch, Bn, v, 8) == plain
    one = dict(w, target=w["target"][:1].cuda().expand(T, V), draft=w["draft"][:1].cuda().expand(T, V))
    same = dict(w, target=w["target"][:1].repeat(T, 1), draft=w["draft"][:1].repeat(T, 1))
    assert run_verify(torch, Bn, one, 8) == check_verify(torch, Bn, same, 8)


def test_verify_bad_rows(torch, Bn):
    """Sequences whose rows break their bounds get nothing; the others are not touched by it."""
    w = walk_inputs(torch, [5, 5, 5], 64, torch.float32, 2, 8, True)
    good = run_verify(torch, Bn, w, 5)
    bad = dict(w, cu=[0, 5, 10, 16])
    got = run_verify(torch, Bn, bad, 5, Bn.IDX_STATUS_BAD_LEN, max_q=6)
    assert [g[:2] for g in got] == [g[:2] for g in good] and got[0][2] == [-1] * 5 and got[1][2] == 0 and got[2][2] == [-1] * 5
    got = run_verify(torch, Bn, dict(w, cu=[0, 5, 3, 15]), 5, Bn.IDX_STATUS_BAD_LEN, max_q=5)
    assert got[1] == [good[1][0], 0, 0]
    assert run_verify(torch, Bn, w, 5, Bn.IDX_STATUS_BAD_LEN, max_q=4)[1] == [0, 0, 0]


def test_verify_emits_the_targets_distribution(torch, Bn):
    """16384 walks over three children drawn from q: chi-square of the first tokens over 6 values, 5 degrees of
    freedom, above 30 with a chance of 1.5e-5. One row of probabilities for all nodes."""
    B, n = 16384, 4
    g = torch.Generator().manual_seed(11)
    p = torch.tensor([[0.4, 0.05, 0.05, 0.3, 0.2, 0.0]])
    q = torch.tensor([[0.1, 0.3, 0.2, 0.1, 0.1, 0.2]])
    w = dict(target=p.cuda().expand(B * n, 6), draft=q.cuda().expand(B * n, 6), parents=[-1, 0, 0, 0] * B,
             tokens=torch.multinomial(q[0], B * n, replacement=True, generator=g).tolist(),
             coins=torch.rand(B * n, generator=g).tolist(), last=torch.rand(B, generator=g).tolist(), cu=[n * b for b in range(B + 1)])
    _, _, out = run_verify(torch, Bn, w, 2)
    got = torch.bincount(torch.tensor([o[0] for o in out]), minlength=6)
    want = p[0].double() * B
    assert got[5] == 0 and float(((got - want) ** 2 / want.clamp(min=1e-9))[:5].sum()) < 30


# ------------------------------------------------------------------------------ compaction

def paths(torch, nq, most, seed, keep=None):
    """Random accepted nodes [B, most] and how many; keep: of these counts."""
    g = torch.Generator().manual_seed(seed)
    path, count = torch.full((len(nq), most), -1, dtype=torch.int32), []
    for b, n in enumerate(nq):
        k = min(n, most, keep[b]) if keep else int(torch.randint(0, min(n, most) + 1, (1,), generator=g))
        path[b, :k] = torch.randperm(n, generator=g)[:k].sort().values.int()
        count.append(k)
    return path, count


def tables(torch, lens, P, seed, extra=2):
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // P) for n in lens]
    perm = torch.randperm(sum(need) + extra, generator=g).int()
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + extra


def run_compact(torch, Bn, kind, pool, P, path, count, lens, nq, table, Hkv=0, D=0, status=0, layers=1, **kw):
    """pool: CPU uint8 [layers, pages, stride]. Compares with the plain form, layer by layer."""
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    i32 = dict(dtype=torch.int32, device="cuda")
    dev, st, new = pool.cuda(), torch.zeros(1, **i32), torch.full((len(lens),), -9, **i32)
    lists = (path.cuda(), torch.tensor(count, **i32), torch.tensor(lens, **i32), torch.tensor(cu, **i32), table.cuda())
    args = dict(layers=layers, layer_stride=dev.stride(0) if layers > 1 else 0, new_lens=new, dev_status=st)
    if kind == "kv":
        Bn.idx_kv_compact(*lists, dev, pool.shape[1], P, dev.stride(1), Hkv, D, **args)
    else:
        Bn.idx_k_compact(*lists, kind, dev, pool.shape[1], P, dev.stride(1), **args)
    got = dev.cpu()
    for layer in range(layers):
        if kind == "kv":
            want, want_new, want_status = dr.kv_compact(pool[layer], Hkv, P, D, path, count, lens, cu, table)
        else:
            want, want_new, want_status = dr.k_compact(pool[layer], kind, P, path, count, lens, cu, table)
        assert int(st) == want_status == status
        assert new.tolist() == want_new
        assert torch.equal(got[layer], want), (got[layer] != want).nonzero()[:5].tolist()


COMPACT = [([5], [5]), ([40, 7, 129, 16], [9, 7, 30, 16]), ([300, 64, 31, 100, 1], [70, 1, 20, 33, 1]),
           ([200, 17, 128, 0, 65], [64, 16, 128, 0, 2])]


def kv_pool(torch, layers, pages, H, P, D, seed, spread, slack=0):
    """Any codes (NaN too) and scales; spread 200: scale bytes that the store does not write."""
    g = torch.Generator().manual_seed(seed)
    pool = torch.randint(0, 256, (layers, pages, H * (2 * P * D + 16) + slack), generator=g).to(torch.uint8)
    for x in pool:
        _, scales = ref.kv_views(x, H, P, D)
        scales.copy_((torch.randint(0, 256, scales.shape, generator=g) if spread == 200 else
                      120 + torch.randint(0, spread + 1, scales.shape, generator=g)).to(torch.uint8))
    return pool


@pytest.mark.parametrize("lens,nq", COMPACT)
@pytest.mark.parametrize("H,D,P,layers,spread", [(1, 64, 64, 1, 3), (3, 128, 128, 2, 1), (5, 64, 128, 1, 12), (4, 128, 64, 1, 200)])
def test_kv_compact(torch, Bn, lens, nq, H, D, P, layers, spread):
    table, pages = tables(torch, lens, P, D)
    pool = kv_pool(torch, layers, pages, H, P, D, H, spread, 32)
    for seed, most in ((0, 5), (1, 20), (2, 130)):
        path, count = paths(torch, nq, most, seed)
        run_compact(torch, Bn, "kv", pool, P, path, count, lens, nq, table, H, D, 0, layers)
    path, count = paths(torch, nq, 128, 3, [1000] * len(nq))  # all of them: nothing moves
    run_compact(torch, Bn, "kv", pool, P, path, count, lens, nq, table, H, D, 0, layers)


@pytest.mark.parametrize("lens,nq", COMPACT)
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("layers", [1, 3])
def test_k_compact(torch, Bn, lens, nq, P, kind, layers):
    table, pages = tables(torch, lens, P, P)
    g = torch.Generator().manual_seed(P)
    pool = torch.randint(0, 256, (layers, pages, (68, 132)[kind] * P + 16), generator=g).to(torch.uint8)
    for seed, most in ((0, 5), (1, 20), (2, 130)):
        path, count = paths(torch, nq, most, seed)
        run_compact(torch, Bn, kind, pool, P, path, count, lens, nq, table, 0, 0, 0, layers)


@pytest.mark.parametrize("kind", ["kv", 0, 1])
def test_compact_odd_inputs(torch, Bn, kind):
    """Refused requests (fewer keys than rows), counts and paths that break their bounds, pages outside the pool."""
    P, H, D = 64, 2, 64
    lens, nq = [100, 100, 100, 100, 2, 100, 100, -1, 100], [6] * 9
    table, pages = tables(torch, lens, P, 1)
    pool = kv_pool(torch, 1, pages, H, P, D, 2, 3)
    run = lambda path, count, status, t=table, ln=lens: run_compact(  # noqa: E731
        torch, Bn, kind, pool, P, path, count, ln, nq, t, H, D, status)
    path, count = paths(torch, nq, 4, 1, [3] * 9)
    ok = [100, 100, 100, 100, 2, 100, 100, 0, 100]
    run(path, count, 0, ln=ok[:7] + [0, 100])
    run(path, count, 0x10)
    run(path, [3, -1, 5, 7, 3, 3, 3, 3, 3], 0x10, ln=ok)
    p = path.clone()
    p[0, 1], p[1, 2], p[2, 0], p[3, 2] = p[0, 0], 6, -1, 1 << 30
    run(p, count, 0x40, ln=ok)
    t = table.clone()
    t[0, 1], t[1, 1] = pages, -3
    t[2] = pages
    run(path, count, 0x4, t, ok)
    run(path, count, 0x10, ln=[100, 100, 100, 100, 2, 100, 100, 1 << 30, 2147483647])


def test_compact_far_pages_and_interleaved_layers(torch, Bn):
    """Layers of a page side by side, and pages behind 2^32 bytes."""
    P, H, D, L = 64, 1, 64, 2
    lens, nq = [40, 70], [12, 9]
    table, pages = tables(torch, lens, P, 3)
    pool = kv_pool(torch, L, pages, H, P, D, 5, 3)
    path, count = paths(torch, nq, 6, 4, [5, 5])
    cu = [0, 12, 21]
    i32 = dict(dtype=torch.int32, device="cuda")
    lists = (path.cuda(), torch.tensor(count, **i32), torch.tensor(lens, **i32), torch.tensor(cu, **i32), table.cuda())
    stride = (1 << 32) // (pages - 1) // 16 * 16 + 4096
    big = torch.zeros(pages, stride, dtype=torch.uint8, device="cuda")
    n = pool.shape[2]
    for layer in range(L):
        big[:, layer * n:(layer + 1) * n] = pool[layer].cuda()
    Bn.idx_kv_compact(*lists, big, pages, P, stride, H, D, layers=L, layer_stride=n)
    for layer in range(L):
        assert torch.equal(big[:, layer * n:(layer + 1) * n].cpu(), dr.kv_compact(pool[layer], H, P, D, path, count, lens, cu, table)[0])


# ------------------------------------------------------------------------------ pages

def run_pages(torch, Bn, s, in_place=False):
    i32 = dict(dtype=torch.int32, device="cuda")
    t = lambda x, *shape: torch.tensor(x, **i32).reshape(shape or (-1,))  # noqa: E731
    n, width, new_width, pages = len(s["parent"]), s["width"], s["new_width"], len(s["shares"])
    blank = [[-9] * new_width for _ in range(n)]
    new_table, new_lens, shares = t(blank, n, new_width), t([-9] * n), t(s["shares"])
    new_shares = shares if in_place else torch.full((pages,), -9, **i32)
    new_free, span, copies, st = t([-9] * s["cap"]), t([-9, -9]), t([[-9, -9]] * n, n, 2), torch.zeros(1, **i32)
    Bn.idx_pages_update(t(s["parent"]), t(s["keep"]), t(s["table"], len(s["lens"]), width), t(s["lens"]), s["P"], new_table, new_lens,
                        shares, new_shares, t(s["free"]), t(s["span"]), new_free, span, copies, dev_status=st)
    want = dr.pages_update(s["parent"], s["keep"], s["table"], s["lens"], s["P"], blank, s["shares"], s["free"], s["span"],
                           [-9] * s["cap"])
    got = (new_table.tolist(), new_lens.tolist(), new_shares.tolist(), new_free.tolist(), span.tolist(), copies.tolist(), int(st))
    for name, x, y in zip(("table", "lens", "shares", "free", "span", "copies", "status"), got, want):
        assert x == y, name
    return got


def page_state(torch, B, n_out, P, most, seed, share=0.5, spare=40, odd=False):
    """Rows that share prefixes at random, forks, cuts, ends; odd: lengths, parents and pages that break their bounds."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=g))  # noqa: E731
    lens = [r(0, most + 1) for _ in range(B)]
    width = -(-max(lens + [0]) // P) + r(0, 2)
    ids = torch.randperm(sum(-(-x // P) for x in lens) + spare, generator=g).tolist()
    table, at = [], 0
    for b in range(B):
        need = -(-lens[b] // P)
        row = ids[at:at + need]
        at += need
        if b and float(torch.rand(1, generator=g)) < share:  # the first full pages are another row's
            other = r(0, b)
            m = r(0, min(lens[b], lens[other]) // P + 1)
            row[:m] = table[other][:m]
        table.append(row + [-5] * (width - need))
    holders = {}
    for b in range(B):
        for page in table[b][:-(-lens[b] // P)]:
            holders[page] = holders.get(page, 0) + 1
    shares = [max(0, holders.get(p, 0) - 1) for p in range(len(ids))]
    free = [p for p in ids if p not in holders]
    parent, keep = [], []
    for _ in range(n_out):
        p = r(-1, B) if B else -1
        k = 0 if p < 0 else r(0, lens[p] + 1) if r(0, 2) else lens[p]
        parent.append(p)
        keep.append(k)
    span = [r(0, 3), len(free)] if len(free) > 3 else [0, len(free)]
    if r(0, 3) == 0:
        span[1] = min(len(free), span[0] + r(0, 4))
    new_width = width + r(0, 3)
    if odd and B and n_out:
        for _ in range(3):
            b = r(0, n_out)
            kind = r(0, 5)
            if kind == 0:
                parent[b] = B + r(0, 9)
            elif kind == 1:
                keep[b] = -1 - r(0, 9)
            elif kind == 2:
                keep[b] = keep[b] + 100000
            elif kind == 3:
                lens[r(0, B)] = (-1, 1 << 30)[r(0, 2)]
            else:
                row = table[r(0, B)]
                if row:
                    row[r(0, len(row))] = (-1, len(ids), 1 << 30)[r(0, 3)]
        if r(0, 4) == 0:
            span = [5, 3]
        if r(0, 4) == 0 and new_width > 1:
            new_width = max(1, width - 1)
        if r(0, 4) == 0 and free:
            free[r(0, len(free))] = len(ids) + 3
    return dict(parent=parent, keep=keep, table=table, lens=lens, P=P, width=width, new_width=new_width, shares=shares, free=free,
                span=span, cap=len(ids) + r(0, 3))


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("B,n_out,P,most", [(1, 1, 64, 200), (5, 9, 64, 500), (40, 33, 128, 1500), (3, 50, 64, 130), (70, 70, 64, 64)])
def test_pages_update(torch, Bn, B, n_out, P, most, seed):
    run_pages(torch, Bn, page_state(torch, B, n_out, P, most, 100 * seed + B), in_place=seed % 2 == 1)


@pytest.mark.parametrize("seed", range(20))
def test_pages_update_odd_inputs(torch, Bn, seed):
    run_pages(torch, Bn, page_state(torch, 9, 14, 64, 400, seed, odd=True), in_place=seed % 2 == 1)


@pytest.mark.parametrize("B,n_out,most,spare", [(1500, 1500, 300, 700), (16384, 16384, 60, 20000), (0, 3, 0, 9), (4, 0, 300, 9), (0, 0, 0, 0),
                                                (2, 5, 20000, 70000)])
def test_pages_update_sizes(torch, Bn, B, n_out, most, spare):
    s = page_state(torch, min(B, 400), min(n_out, 400), 64, most, 7, spare=spare)
    if B > 400:  # the same rows again, each a holder of its pages
        k = B // 400 + 1
        s["table"], s["lens"] = (s["table"] * k)[:B], (s["lens"] * k)[:B]
        s["shares"] = _count(s)
        s["parent"] = [p if p < 0 else (p + 400 * (b % k)) % B for b, p in enumerate((s["parent"] * k)[:n_out])]
        s["keep"] = [0 if p < 0 else min(x, s["lens"][p]) for p, x in zip(s["parent"], (s["keep"] * k)[:n_out])]
    run_pages(torch, Bn, s)


def _count(s):
    holders = [0] * len(s["shares"])
    for row, n in zip(s["table"], s["lens"]):
        for page in row[:-(-n // s["P"])]:
            holders[page] += 1
    return [max(0, h - 1) for h in holders]


def test_pages_update_excess_release(torch, Bn):
    """Counts that say less than the tables: the page becomes free once, and the status word tells."""
    s = dict(parent=[], keep=[], table=[[1, 2], [1, 3]], lens=[100, 100], P=64, width=2, new_width=1, shares=[0] * 6, free=[4, 5],
             span=[0, 2], cap=6)
    got = run_pages(torch, Bn, s)
    assert got[-1] == Bn.IDX_STATUS_BAD_PAGE and got[3][:5] == [4, 5, 1, 2, 3]


def test_pages_feed_calls_that_read_before_they_wait(torch, Bn):
    """The top-k reads lengths before it waits for the kernel in front of it: a replayed graph of the update and the
    top-k sees each step's new lengths."""
    B, P, L = 64, 64, 512
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.arange(B * 8, **i32).reshape(B, 8).contiguous(), torch.full((B,), L, **i32)
    parent, keep = torch.arange(B, **i32), torch.full((B,), L, **i32)
    new_table, new_lens, shares = torch.zeros_like(table), torch.zeros_like(lens), torch.zeros(B * 8, **i32)
    new_shares, free, span = torch.zeros_like(shares), torch.zeros(1, **i32), torch.zeros(2, **i32)
    new_free, new_span, copies = torch.zeros_like(shares), torch.zeros(2, **i32), torch.zeros(B, 2, **i32)
    logits, idx = torch.arange(L, device="cuda").float().repeat(B, 1).contiguous(), torch.zeros(B, 4, **i32)
    cu = torch.arange(B + 1, **i32)

    def step():
        Bn.idx_pages_update(parent, keep, table, lens, P, new_table, new_lens, shares, new_shares, free, span, new_free, new_span, copies)
        Bn.idx_topk(logits, new_lens, cu, 0, L, 4, idx)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in (5, 100, 17, 511, 4):
        keep.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        assert all(sorted(r) == [n - 4, n - 3, n - 2, n - 1] for r in idx.tolist()), n


@pytest.mark.parametrize("n,layers,page,slack", [(1, 1, 16, 0), (5, 3, 8208, 16), (40, 1, 4352, 0), (3, 2, 1 << 20, 48), (200, 4, 65568, 0)])
def test_pages_copy(torch, Bn, n, layers, page, slack):
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = 2 * n + 1
    pool = torch.randint(0, 256, (layers, pages, page + slack), generator=g, device="cuda", dtype=torch.uint8)
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    pairs = torch.stack([perm[:n], perm[n:2 * n]], 1)
    pairs[1::3] = -1
    if n > 4:
        pairs[4, 1] = pairs[4, 0]
        pairs[3, 0] = -1
    want = pool.clone()
    ok = (pairs >= 0).all(1) & (pairs[:, 0] != pairs[:, 1])
    src, dst = pairs[ok].long().unbind(1)
    want[:, dst, :page] = pool[:, src, :page]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Bn.idx_pages_copy(pairs.contiguous(), pool, pages, page, page + slack, layers=layers, layer_stride=pool.stride(0), dev_status=st)
    assert int(st) == 0 and torch.equal(pool, want)
    bad = torch.tensor([[0, pages], [pages, 1], [1 << 30, 0]], dtype=torch.int32, device="cuda")
    Bn.idx_pages_copy(bad, pool, pages, page, page + slack, layers=layers, layer_stride=pool.stride(0), dev_status=st)
    assert int(st) == Bn.IDX_STATUS_BAD_PAGE and torch.equal(pool, want)


def test_pages_copy_far_pages(torch, Bn):
    stride = (1 << 31) + 4096
    pool = torch.zeros(3 * stride, dtype=torch.uint8, device="cuda")
    pool[:8192].random_(0, 256)
    Bn.idx_pages_copy(torch.tensor([[0, 2]], dtype=torch.int32, device="cuda"), pool, 3, 8192, stride)
    assert torch.equal(pool[2 * stride:2 * stride + 8192], pool[:8192]) and not pool[8192:2 * stride].any()


# ------------------------------------------------------------------------------ all of them together

@pytest.mark.parametrize("Hq,Hkv,D,P,nodes,k", [(8, 2, 64, 64, 7, 0), (16, 1, 128, 64, 12, 0), (16, 1, 64, 128, 5, 40)])
def test_drafting_steps(torch, Bn, Hq, Hkv, D, P, nodes, k):
    """Steps of a serving loop: metadata, store, attention of the trees, verification, compaction, page rows, copies. Some
    requests fork, some end. The cache that each row sees is rebuilt from what was stored, token by token, and the attention is
    held to the plain form over it; pages are neither lost nor held twice."""
    g = torch.Generator().manual_seed(nodes + k)
    i32 = dict(dtype=torch.int32, device="cuda")
    B, V, width, pages = 6, 50, 6, 60
    hb = Hkv * (2 * P * D + 16)
    pool = torch.zeros(pages, hb, dtype=torch.uint8, device="cuda")
    free, span = torch.randperm(pages, generator=g).int().cuda(), torch.tensor([0, pages], **i32)
    shares, table = torch.zeros(pages, **i32), torch.full((B, width), -1, **i32)
    ctx = torch.tensor([0, 30, 61, 64, 100, 17], **i32)
    status = torch.zeros(1, **i32)
    dt = torch.float16
    # prompts
    cu, lens = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)

    def meta(ctx, new, T):
        pos, slots, nxt = torch.zeros(T, **i32), torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(1, **i32)
        Bn.idx_step_meta(ctx, new, table, P, width * P, free, span, pages, cu, lens, pos, slots, nxt, dev_status=status)
        span[0] = nxt[0]
        return slots

    T = int(ctx.sum())
    kv = torch.randn(T, 2, Hkv, D, generator=g).to(dt).cuda()
    slots = meta(torch.zeros(B, **i32), ctx, T)
    Bn.idx_kv_store(kv[:, 0], kv[:, 1], slots, pool, pages, P, hb, dev_status=status)
    codes, scales = ref.kv_views(pool, Hkv, P, D)
    for step in range(5):
        T = B * nodes
        slots = meta(ctx, torch.full((B,), nodes, **i32), T)
        kv = torch.randn(T, 2, Hkv, D, generator=g).to(dt).cuda() * (step + 1)
        Bn.idx_kv_store(kv[:, 0], kv[:, 1], slots, pool, pages, P, hb, dev_status=status)
        parents = sum((dr.random_tree(nodes, g, 3) for _ in range(B)), [])
        sets = sum((dr.ancestors(parents[b * nodes:(b + 1) * nodes]) for b in range(B)), [])
        mask = dr.mask_words(sets, 1).cuda()
        q = torch.randn(T, Hq, D, generator=g).to(dt).cuda()
        out, lse = torch.zeros_like(q), torch.zeros(T, Hq, device="cuda")
        hl = lens.tolist()
        sel = None
        if k:
            sel = torch.stack([torch.randperm(max(k, hl[t // nodes] - nodes), generator=g)[:k] for t in range(T)]).int().cuda()
        Bn.idx_attn_tree(q, pool, pages, P, hb, Hkv, table, lens, cu, mask, nodes, width * P, D ** -0.5, out, lse=lse, sel_idx=sel,
                         dev_status=status)
        keys = dr.keys_of(sets, [nodes] * B, hl, T, sel).cuda()
        o, l, otol, ltol = ref.attention(q, pool, P, Hkv, table, hl, cu.tolist(), 0, D ** -0.5, keys)
        assert ((out.double() - o).abs() <= otol).all()
        # verification
        target = (torch.randn(T, V, generator=g) * 2).softmax(-1)
        draft = (target.log() * 0.7).softmax(-1)
        tokens = [int(torch.multinomial(draft[t - t % nodes + max(parents[t], 0)], 1, generator=g)) for t in range(T)]
        coins, last = torch.rand(T, generator=g), torch.rand(B, generator=g)
        path, n_path, emitted = torch.zeros(B, 5, **i32), torch.zeros(B, **i32), torch.zeros(B, 5, **i32)
        Bn.idx_draft_verify(target.cuda(), draft.cuda(), torch.tensor(tokens, **i32), torch.tensor(parents, **i32), coins.cuda(),
                            last.cuda(), cu, nodes, path, n_path, emitted, dev_status=status)
        want = dr.verify(target, draft, tokens, parents, coins.tolist(), last.tolist(), cu.tolist(), 5)
        assert (path.tolist(), n_path.tolist(), emitted.tolist()) == want[:3]
        # compaction: each kept token's values are what they were, rounded once more at most
        before, table_was = pool.clone(), table.cpu()
        new_lens = torch.zeros(B, **i32)
        Bn.idx_kv_compact(path, n_path, lens, cu, table, pool, pages, P, hb, Hkv, D, new_lens=new_lens, dev_status=status)
        plain, plain_lens, _ = dr.kv_compact(before.cpu(), Hkv, P, D, path.cpu(), n_path.tolist(), hl, cu.tolist(), table_was)
        assert torch.equal(pool.cpu(), plain) and new_lens.tolist() == plain_lens
        # page rows: row 0 forks over the last row, one row ends and a new one begins every other step
        parent, keep = list(range(B)), new_lens.tolist()
        parent[B - 1], keep[B - 1] = 0, keep[0]
        if step % 2:
            parent[2], keep[2] = -1, 0
        new_table, next_lens, new_shares = torch.full_like(table, -1), torch.zeros(B, **i32), torch.zeros_like(shares)
        new_free, new_span, copies = torch.zeros(pages, **i32), torch.zeros(2, **i32), torch.zeros(B, 2, **i32)
        Bn.idx_pages_update(torch.tensor(parent, **i32), torch.tensor(keep, **i32), table, lens, P, new_table, next_lens, shares,
                            new_shares, free, span, new_free, new_span, copies, dev_status=status)
        Bn.idx_pages_copy(copies, pool, pages, hb, hb, dev_status=status)
        table, shares, free, span, ctx = new_table, new_shares, new_free, new_span, next_lens
        assert int(status) == 0 and ctx.tolist() == keep
        held = [p for row, n in zip(table.tolist(), keep) for p in row[:-(-n // P)]]
        loose = free[:int(span[1])].tolist()
        assert sorted(set(held) | set(loose)) == list(range(pages)) and not set(held) & set(loose) and len(set(loose)) == len(loose)
        assert [held.count(p) - 1 if p in held else 0 for p in range(pages)] == shares.tolist()
        ends = [row[n // P] for row, n in zip(table.tolist(), keep) if n % P]
        assert all(held.count(p) == 1 for p in ends)
        # a fork reads what its parent holds
        n = keep[0]
        pos = torch.arange(n, device="cuda")
        a, b = table[0, pos // P].long(), table[B - 1, pos // P].long()
        assert torch.equal(codes[a, :, pos % P], codes[b, :, pos % P])
