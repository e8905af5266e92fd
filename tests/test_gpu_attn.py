"""The step metadata, the 8-bit KV store and the paged attention on the GPU against plain 64-bit
forms (tests/attn_ref.py): bytes and whole numbers bit for bit, attention within bounds derived
there from the arithmetic."""
import itertools
import math

import pytest

import attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as T
    from sparse_attention_indexer_mqa_gb300 import binding
    binding.load()
    return T


@pytest.fixture(scope="module")
def Bn():
    from sparse_attention_indexer_mqa_gb300 import binding
    return binding


# ------------------------------------------------------------------------------ step metadata

def run_meta(torch, Bn, ctx, new, P, longest, free, span, num_pages, cap, width, seed=0, status_want=None):
    g = torch.Generator().manual_seed(seed)
    B = len(ctx)
    table = [[int(x) for x in torch.randint(0, num_pages, (width,), generator=g)] for _ in range(B)]
    i32 = dict(dtype=torch.int32, device="cuda")
    t = torch.tensor(table, **i32).reshape(B, width)
    cu, lens = torch.full((B + 1,), -9, **i32), torch.full((B,), -9, **i32)
    pos, slots = torch.full((cap,), -9, **i32), torch.full((cap,), -9, dtype=torch.int64, device="cuda")
    nxt, status = torch.full((1,), -9, **i32), torch.zeros(1, **i32)
    Bn.idx_step_meta(torch.tensor(ctx, **i32), torch.tensor(new, **i32), t, P, longest, torch.tensor(free, **i32),
                     torch.tensor(span, **i32), num_pages, cu, lens, pos, slots, nxt, dev_status=status)
    want = ref.step_meta(ctx, new, table, P, longest, free, span, num_pages, cap)
    got = (t.tolist(), cu.tolist(), lens.tolist(), pos.tolist(), slots.tolist(), int(nxt), int(status))
    for name, x, y in zip(("table", "cu", "lens", "pos", "slots", "next", "status"), got, want):
        assert x == y, name
    if status_want is not None:
        assert got[-1] == status_want


@pytest.mark.parametrize("B,P,q_hi,ctx_hi,cap_extra", [
    (1, 64, 1, 1, 0), (64, 128, 1, 9000, 0), (64, 64, 300, 700, 9), (257, 64, 40, 500, 0), (300, 128, 5, 200, 1000),
    (5, 128, 9000, 0, 0), (4097, 64, 3, 130, 1), (16384, 64, 1, 64, 0)])
def test_meta(torch, Bn, B, P, q_hi, ctx_hi, cap_extra):
    g = torch.Generator().manual_seed(B)
    ctx = torch.randint(0, ctx_hi + 1, (B,), generator=g).tolist()
    new = torch.randint(0, q_hi + 1, (B,), generator=g).tolist()
    longest = max(a + b for a, b in zip(ctx, new))
    width = -(-longest // P) + 1
    need = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(ctx, new))
    pages = 4 * B + need
    free = torch.randperm(pages, generator=g)[:need + 5].tolist()
    run_meta(torch, Bn, ctx, new, P, longest, free, [3, 3 + need], pages, sum(new) + cap_extra, width, B, 0)


def test_meta_refused_requests(torch, Bn):
    """Too few pages, lengths that break their bounds, rows past the capacity, bad page ids."""
    free = list(range(20, 30))
    a = (torch, Bn)
    run_meta(*a, [64, 0, 10, 63], [1, 130, 5, 1], 64, 256, free, [0, 3], 64, 137, 4, 1, 0x20)
    run_meta(*a, [64, 0, 64], [1, 0, 1], 64, 256, free, [10, 10], 64, 9, 4, 2, 0x20)
    run_meta(*a, [-1, 5, 200, 3], [4, -2, 60, 7], 64, 256, free, [0, 10], 64, 80, 4, 3, 0x10)
    run_meta(*a, [0, 0, 0, 5], [10, 10, 10, 0], 64, 256, free, [0, 10], 64, 25, 4, 4, 0x10)
    run_meta(*a, [0, 70], [3, 3], 64, 256, free, [4, 11], 64, 6, 4, 5, 0x24)
    run_meta(*a, [0, 70], [3, 3], 64, 256, free, [-1, 5], 64, 6, 4, 5, 0x24)
    run_meta(*a, [0, 0], [3, 3], 64, 256, [7, -5, 900], [0, 3], 64, 6, 4, 6, 0x4)
    run_meta(*a, [2147483647, 0], [2147483647, 3], 64, 256, free, [0, 3], 64, 6, 4, 7, 0x10)
    run_meta(*a, [1, 2], [0, 0], 64, 256, free, [2, 5], 64, 0, 4, 8, 0)
    run_meta(*a, [], [], 64, 0, free, [2, 5], 64, 4, 1, 9, 0)


def test_meta_feeds_calls_that_read_before_they_wait(torch, Bn):
    """The scorer and the top-k read lengths and the page table before they wait for the kernel
    before them: a replayed graph of metadata and top-k must see each step's new lengths."""
    B, P, L = 64, 64, 512
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new = torch.zeros(B, **i32), torch.ones(B, **i32)
    table = torch.arange(B * 8, **i32).reshape(B, 8).contiguous()
    cu, lens, pos = torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    slots, nxt = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(1, **i32)
    span, free = torch.tensor([0, 4 * B], **i32), torch.arange(4 * B, **i32)
    logits = torch.arange(L, device="cuda").float().repeat(B, 1).contiguous()
    idx = torch.zeros(B, 4, **i32)

    def step():
        Bn.idx_step_meta(ctx, new, table, P, L, free, span, 8 * B, cu, lens, pos, slots, nxt)
        Bn.idx_topk(logits, lens, cu, 0, L, 4, idx)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in (5, 100, 17, 511, 4):
        ctx.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        # the top-k's order: above the k-th value in index order, then the k-th
        assert idx.tolist() == [[n - 2, n - 1, n, n - 3]] * B, n


# ------------------------------------------------------------------------------ store

def make_rows(torch, n, H, D, dt, seed, spread=6.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 2, H, D, generator=g) * torch.exp2((torch.rand(n, 2, H, 1, generator=g) - 0.5) * 2 * spread)
    return x.to(dt)


def run_store(torch, Bn, pool, kv, slots, P, status_want=0, offset=0):
    dev = pool.cuda()
    d = kv.cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Bn.idx_kv_store(d[:, 0], d[:, 1], torch.tensor(slots, dtype=torch.int64, device="cuda"), dev, pool.shape[0], P,
                    pool.stride(0), dev_status=st)
    want = ref.store(pool, kv[:, 0], kv[:, 1], torch.tensor(slots, dtype=torch.int64), P)
    got = dev.cpu()
    assert int(st) == status_want
    assert torch.equal(got, want)
    return got


def empty_pool(torch, pages, H, D, P, seed=0, slack=0):
    """A pool of arbitrary bytes (the store has to leave what is not its own alone)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (pages, H * (2 * P * D + 16) + slack), generator=g).to(torch.uint8)


@pytest.mark.parametrize("H,D,P,dt,ctx,new", [
    (1, 64, 64, "bfloat16", [0], [1]), (1, 128, 128, "float16", [0, 15, 16, 17, 100], [1, 1, 1, 1, 1]),
    (3, 64, 128, "float16", [0, 5, 120], [130, 30, 9]), (8, 128, 64, "bfloat16", [0, 63, 1], [200, 2, 64]),
    (5, 128, 128, "bfloat16", [33] * 7, [1, 2, 3, 14, 15, 16, 17])])
def test_store(torch, Bn, H, D, P, dt, ctx, new):
    dt = getattr(torch, dt)
    pages = sum(-(-(a + b) // P) for a, b in zip(ctx, new)) + 2
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(7)).tolist()
    pool = empty_pool(torch, pages, H, D, P, 1, 32)
    at, old, slots = 0, [], []
    for a, b in zip(ctx, new):
        n = -(-(a + b) // P)
        own = [perm[at + p // P] * P + p % P for p in range(a + b)]
        old += own[:a]
        slots += own[a:]
        at += n
    if old:  # what was there before, by the store itself
        pool = run_store(torch, Bn, pool, make_rows(torch, len(old), H, D, dt, 2), old, P)
    pool = run_store(torch, Bn, pool, make_rows(torch, len(slots), H, D, dt, 3), slots, P)
    run_store(torch, Bn, pool, make_rows(torch, len(slots), H, D, dt, 3), slots, P)  # again: the same


def test_store_token_by_token_equals_at_once(torch, Bn):
    """Appending rescales the kept codes by powers of two: but for subnormal codes, a block that
    grows token by token ends as if stored at once. Values without tiny ones: bit for bit."""
    H, D, P = 2, 64, 64
    g = torch.Generator().manual_seed(5)
    kv = (torch.rand(40, 2, H, D, generator=g) + 0.5) * torch.exp2(torch.randint(-1, 2, (40, 2, H, 1), generator=g))
    kv = kv.to(torch.bfloat16)
    whole = run_store(torch, Bn, empty_pool(torch, 1, H, D, P), kv, list(range(40)), P)
    step = empty_pool(torch, 1, H, D, P)
    for i in range(40):
        step = run_store(torch, Bn, step, kv[i:i + 1], [i], P)
    assert torch.equal(whole, step)


def test_store_rolls_back_and_starts_afresh(torch, Bn):
    H, D, P, bf = 1, 128, 64, torch.bfloat16
    pool = run_store(torch, Bn, empty_pool(torch, 2, H, D, P), make_rows(torch, 30, H, D, bf, 1) * 64, list(range(30)), P)
    pool = run_store(torch, Bn, pool, make_rows(torch, 3, H, D, bf, 2), [20, 21, 22], P)    # keeps 16 .. 19
    pool = run_store(torch, Bn, pool, make_rows(torch, 4, H, D, bf, 3) * 2 ** -9, [16, 17, 18, 19], P)  # afresh
    run_store(torch, Bn, pool, make_rows(torch, 2, H, D, bf, 4), [3, 9], P)  # gaps are allowed


@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
def test_store_extreme_values(torch, Bn, dt):
    H, D, P, dt = 2, 64, 64, getattr(torch, dt)
    big = torch.finfo(dt).max
    kv = make_rows(torch, 64, H, D, dt, 9, 3.0)
    kv[0, 0, 0, :8] = torch.tensor([math.inf, -math.inf, 0.0, -0.0, 1e-7, -1e-7, 448.0, 449.0]).to(dt)
    kv[17, 1, 1, :] = 0.0
    kv[16:32, 0, 0] = 0.0
    kv[32, 0, 1, 3] = big
    kv[33, 0, 1, 4] = -big
    kv[48, 1, 0, :] = torch.finfo(dt).tiny
    kv[49:64, 1, 0, :] = torch.finfo(dt).tiny / 4
    pool = empty_pool(torch, 1, H, D, P)
    run_store(torch, Bn, pool, kv, list(range(64)), P)
    kv[5, 1, 1, 7] = math.nan
    kv[6, 0, 0, :] = math.nan
    run_store(torch, Bn, pool, kv, list(range(64)), P, 0x40)
    # exactly at, and just above, the largest code times a power of two
    kv = torch.zeros(64, 2, H, D, dtype=dt)
    for i, x in enumerate([448.0, 450.0, 1.75, 1.7578125]):
        kv[16 * i, :, :, 0] = x
        kv[16 * i + 1, :, :, :] = torch.linspace(-1, 1, D).to(dt)
    run_store(torch, Bn, pool, kv, list(range(64)), P)


def test_store_skips_and_flags(torch, Bn):
    H, D, P, bf = 1, 64, 64, torch.bfloat16
    pool = empty_pool(torch, 2, H, D, P)
    rows = lambda n: make_rows(torch, n, H, D, bf, n)
    run_store(torch, Bn, pool, rows(6), [-1, 0, -1, 16, 17, -1], P)
    run_store(torch, Bn, pool, rows(3), [128, 5, 1 << 40], P, 0x1)
    run_store(torch, Bn, pool, rows(4), [5, 5, 6, 20], P, 0x1)       # the same slot twice
    run_store(torch, Bn, pool, rows(3), [9, 8, 40], P, 0x1)          # not increasing
    run_store(torch, Bn, pool, rows(0), [], P)


def test_store_far_pages(torch, Bn):
    """Pages past 2^32 bytes of the pool."""
    H, D, P = 1, 64, 64
    stride = 1 << 28
    pool = torch.zeros(18, stride, dtype=torch.uint8, device="cuda")
    kv = make_rows(torch, 2, H, D, torch.bfloat16, 3).cuda()
    for page in (7, 8, 15, 16, 17):
        s = torch.tensor([page * P + 3, page * P + 40], device="cuda")
        Bn.idx_kv_store(kv[:, 0], kv[:, 1], s, pool, 18, P, stride)
        want = ref.store(torch.zeros(1, 2 * P * D + 16, dtype=torch.uint8), kv[:, 0].cpu(), kv[:, 1].cpu(),
                         torch.tensor([3, 40]), P)
        assert torch.equal(pool[page, :2 * P * D + 16].cpu(), want[0])


# ------------------------------------------------------------------------------ attention

class Att:
    """Inputs of an attention call: a filled cache with stale NaN codes past every length."""

    def __init__(self, torch, lens, nq, Hq, Hkv, D, P, dt, seed=0, pad=0, spread=1, width_extra=1, stride_extra=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.lens, self.nq = torch, lens, nq
        self.Hq, self.Hkv, self.D, self.P = Hq, Hkv, D, P
        need = [-(-n // P) for n in lens]
        self.pages = sum(need) + 1
        perm = torch.randperm(self.pages, device="cuda", generator=g).int()
        self.table = torch.full((len(lens), max(need + [0]) + width_extra), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.pool = torch.full((self.pages, Hkv * (2 * P * D + 16) + stride_extra), 0x7F, dtype=torch.uint8,
                               device="cuda")
        codes, scales = ref.kv_views(self.pool, Hkv, P, D)
        scales.fill_(255)
        for b, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            page = self.table[b, pos // P].long()
            x = torch.randn(n, Hkv, 2, D, device="cuda", generator=g) * 100
            codes[page, :, pos % P] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            e = torch.randint(120 - spread, 121 + spread, (-(-n // 16), Hkv, 2), device="cuda", generator=g)
            first = pos[::16]
            scales[self.table[b, first // P].long(), :, first % P // 16] = e.to(torch.uint8)
        self.cu = [0]
        for n in nq:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1] + pad
        self.q = torch.randn(self.T, Hq, D, device="cuda", generator=g).to(dt)
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dev_cu = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5
        self.out = torch.full((self.T, Hq, D), 77.0, dtype=dt, device="cuda")
        self.lse = torch.full((self.T, Hq), 77.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, Bn, causal, sel=None, ws=None, **kw):
        args = dict(lse=self.lse, sel_idx=sel, workspace=ws, dev_status=self.status)
        args.update(kw)
        Bn.idx_attn_paged(self.q, self.pool, self.pages, self.P, self.pool.stride(0), self.Hkv, self.table,
                          self.dev_lens, self.dev_cu, causal, max(self.nq), max(self.lens), self.scale, self.out, **args)

    def workspace(self, Bn, n_sel=0):
        n = Bn.idx_attn_workspace_bytes(self.T, self.Hq, self.Hkv, self.D, len(self.lens), max(self.nq),
                                        max(self.lens), n_sel)
        return self.torch.full((max(n, 256),), 255, dtype=self.torch.uint8, device="cuda")

    def check(self, causal, sel=None, status=0):
        torch = self.torch
        o, l, otol, ltol = ref.attention(self.q, self.pool, self.P, self.Hkv, self.table, self.lens, self.cu, causal,
                                         self.scale, sel)
        own = ~torch.isnan(l)
        assert int(self.status) == status
        assert (self.out[~own] == 77).all() and (self.lse[~own] == 77).all(), "rows of no sequence were written"
        got, gl = self.out.double(), self.lse.double()
        assert torch.isfinite(got[own]).all()
        bad = (got - o).abs() > otol
        bad[~own] = False
        assert not bad.any(), (bad.nonzero()[:5].tolist(), float(((got - o).abs() / otol)[own].nan_to_num().max()))
        empty = own & (l == -math.inf)
        assert (gl[empty] == -math.inf).all() and (got[empty] == 0).all()
        full = own & ~empty
        assert ((gl - l).abs()[full] <= ltol[full]).all(), float(((gl - l).abs() / ltol)[full].max())


HEADS = [(1, 1), (4, 1), (7, 1), (8, 2), (12, 4), (16, 1), (34, 2), (64, 1), (128, 1), (136, 1)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("D,P,dt", [(64, 64, "float16"), (128, 128, "bfloat16"), (128, 64, "float16")])
def test_decode(torch, Bn, Hq, Hkv, D, P, dt):
    a = Att(torch, [1, 15, 16, 17, 64, 129, 500, 0, 777], [1] * 9, Hq, Hkv, D, P, getattr(torch, dt), Hq, pad=2)
    a.call(Bn, 0, ws=a.workspace(Bn))
    a.check(0)
    a.out.fill_(77)
    a.lse.fill_(77)
    a.call(Bn, 1)  # no workspace: no split
    a.check(1)


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("D,P,dt", [(64, 128, "bfloat16"), (128, 64, "bfloat16"), (128, 128, "float16")])
@pytest.mark.parametrize("causal", [0, 1])
def test_chunks(torch, Bn, Hq, Hkv, D, P, dt, causal):
    """Ragged chunks; sequences shorter than their queries (rows that see nothing), of no key, of
    no query; rows behind the last sequence."""
    a = Att(torch, [40, 129, 300, 7, 0, 65, 128], [40, 3, 37, 12, 5, 0, 128], Hq, Hkv, D, P, getattr(torch, dt), Hq, pad=3)
    a.call(Bn, causal, ws=a.workspace(Bn))
    a.check(causal)


def lists(torch, a, causal, k, seed=0):
    """Per row: distinct visible keys in any order, then duplicates of some, keys it does not see and
    negative ones mixed in."""
    g = torch.Generator().manual_seed(seed)
    sel = torch.full((a.T, k), -1, dtype=torch.int32)
    for b, n in enumerate(a.lens):
        for i, v in enumerate(ref.visible(n, a.nq[b], causal)):
            ids = torch.randperm(v, generator=g)[:max(0, k - 5)]
            junk = torch.tensor([-1, v, n, 2147483647, -2147483648])
            if len(ids):
                junk[0] = ids[0]
            row = torch.cat([ids, junk])
            row = row[torch.randperm(len(row), generator=g)][:k]
            sel[a.cu[b] + i, :len(row)] = row.int()
    return sel.cuda()


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("D,P,dt", [(64, 64, "bfloat16"), (128, 128, "float16"), (128, 64, "bfloat16")])
@pytest.mark.parametrize("k", [6, 48, 257])
def test_selected(torch, Bn, Hq, Hkv, D, P, dt, k):
    a = Att(torch, [1, 30, 300, 700, 0, 9, 64], [1, 2, 5, 1, 2, 12, 1], Hq, Hkv, D, P, getattr(torch, dt), k + Hq, pad=2)
    sel = lists(torch, a, 1, k)
    a.call(Bn, 1, sel, a.workspace(Bn, k))
    a.check(1, sel)
    a.out.fill_(77)
    a.lse.fill_(77)
    wide = torch.full((a.T, k + 9), 3, dtype=torch.int32, device="cuda")
    wide[:, :k] = sel
    a.call(Bn, 1, wide[:, :k])  # strided rows, no workspace
    a.check(1, sel)


def test_every_key_listed_is_the_dense_result(torch, Bn):
    a = Att(torch, [130, 77], [1, 1], 8, 1, 128, 64, torch.float16)
    sel = torch.arange(130, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    a.call(Bn, 0, sel)
    a.check(0)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (64, 1, 128), (12, 4, 64), (128, 1, 64)])
def test_long_and_split(torch, Bn, Hq, Hkv, D):
    """A key axis that is split, and the same without a workspace; same call, same bits."""
    a = Att(torch, [20011, 4097], [1, 2], Hq, Hkv, D, 64, torch.bfloat16)
    ws = a.workspace(Bn)
    assert ws.numel() > 256
    a.call(Bn, 1, ws=ws)
    a.check(1)
    first, l1 = a.out.clone(), a.lse.clone()
    ws.fill_(0)
    a.call(Bn, 1, ws=ws)
    assert torch.equal(first, a.out) and torch.equal(l1, a.lse)
    a.call(Bn, 1, ws=ws[:ws.numel() // 3 // 256 * 256])
    a.check(1)
    a.call(Bn, 1)
    a.check(1)


@pytest.mark.parametrize("Hq,Hkv,D,B", [(63, 1, 64, 21), (64, 8, 128, 21), (33, 1, 128, 41)])
def test_many_rows_split(torch, Bn, Hq, Hkv, D, B):
    """Enough rows for a join of a warp a row: an odd number of them, padded ones, sequences of no and one key."""
    a = Att(torch, [0, 1, 2600] + [1500 + 37 * i for i in range(B - 3)], [1] * B, Hq, Hkv, D, 64, torch.float16, pad=4)
    ws = a.workspace(Bn)
    assert ws.numel() > 256 and a.T * Hq > 1216
    a.call(Bn, 1, ws=ws)
    a.check(1)
    a.dev_lens[2] = 1 << 30  # refused: none of its rows is written
    a.out[2], a.lse[2] = 77, 77
    kept = a.out.clone()
    a.call(Bn, 1, ws=ws)
    assert torch.equal(a.out, kept) and (a.lse[2] == 77).all() and int(a.status) == Bn.IDX_STATUS_BAD_LEN


def test_full_grids_are_not_split(torch, Bn):
    """Partial results of tiles of many rows cost more than another round of them: prompts that fill the GPU ask for no
    workspace, uneven chunks and short ones on long caches do."""
    assert Bn.idx_attn_workspace_bytes(1024, 32, 8, 128, 1, 1024, 1024) == 0
    assert Bn.idx_attn_workspace_bytes(4096, 32, 8, 128, 4, 1024, 16384) == 0
    assert Bn.idx_attn_workspace_bytes(900, 12, 4, 64, 8, 301, 3300) > 0
    assert Bn.idx_attn_workspace_bytes(128, 32, 8, 128, 1, 128, 16384) > 0


@pytest.mark.parametrize("Hq,nq", [(8, 1), (64, 1), (16, 40)])
def test_block_scales_far_apart(torch, Bn, Hq, nq):
    """V blocks whose scales differ by 2^30 and logits that favour the small ones."""
    a = Att(torch, [320, 100], [nq, nq], Hq, 1, 128, 64, torch.float16, 3, spread=15)
    a.scale = 0.002
    a.call(Bn, 1, ws=a.workspace(Bn))
    a.check(1)


@pytest.mark.parametrize("Hq,nq,sel_k", [(8, 1, 0), (16, 1, 30), (64, 1, 0), (64, 3, 30), (8, 33, 0)])
def test_non_finite_queries_stay_in_their_rows(torch, Bn, Hq, nq, sel_k):
    a = Att(torch, [100, 90], [nq, nq], Hq, 1, 128, 64, torch.bfloat16)
    sel = lists(torch, a, 1, sel_k) if sel_k else None
    clean = a.q.clone()
    a.q[0, 1, 5] = math.nan
    a.q[a.T - 1, Hq - 1, 0] = math.inf
    a.call(Bn, 1, sel)
    mask = torch.zeros(a.T, Hq, dtype=torch.bool, device="cuda")
    mask[0, 1] = mask[a.T - 1, Hq - 1] = True
    assert torch.isnan(a.out[mask]).all() and torch.isnan(a.lse[mask]).all()
    a.q = clean
    o, l, otol, ltol = ref.attention(a.q, a.pool, 64, 1, a.table, a.lens, a.cu, 1, a.scale, sel)
    assert ((a.out.double() - o).abs()[~mask] <= otol[~mask]).all()


@pytest.mark.parametrize("Hq,nq", [(4, 1), (64, 1), (4, 70)])
def test_tiny_and_huge_queries(torch, Bn, Hq, nq):
    """Rows of q over bf16's range of magnitudes, among them zeros and subnormals."""
    a = Att(torch, [200], [nq], Hq, 1, 64, 64, torch.bfloat16)
    for i, f in enumerate([0.0, 1e-39, 1e-30, 30.0]):
        a.q[:, i] *= f
    a.call(Bn, 1)
    a.check(1)


def test_strides(torch, Bn):
    """q as a slice of a wider projection, out with a row stride of its own, a padded pool."""
    for Hq, nq in ((8, 1), (64, 1), (8, 50)):
        a = Att(torch, [150, 40], [nq, nq], Hq, 2, 64, 64, torch.float16, stride_extra=48)
        wide = torch.randn(a.T, 3, Hq, 64, device="cuda").half()
        wide[:, 1] = a.q
        a.q = wide[:, 1]
        big = torch.full((a.T, Hq + 2, 64), 77.0, device="cuda").half()
        a.out = big[:, 1:-1]
        a.call(Bn, 1)
        a.check(1)
        assert (big[:, 0] == 77).all() and (big[:, -1] == 77).all()
        # heads first: [Hq, T, D] seen as [T, Hq, D]
        a.q = a.q.transpose(0, 1).contiguous().transpose(0, 1)
        a.out = torch.full((Hq, a.T, 64), 77.0, device="cuda").half().transpose(0, 1)
        a.call(Bn, 1)
        a.check(1)


@pytest.mark.parametrize("Hq,nq,k", [(8, 1, 0), (64, 1, 0), (8, 40, 0), (8, 1, 20), (64, 2, 20)])
def test_bad_pages_and_lengths(torch, Bn, Hq, nq, k):
    a = Att(torch, [200, 100, 150, 64], [nq] * 4, Hq, 1, 128, 64, torch.bfloat16)
    sel = lists(torch, a, 1, k) if k else None
    good = a.table.clone()
    a.call(Bn, 1, sel)
    a.check(1, sel)
    before = a.out.clone()
    # keys of a page outside the pool count as not there
    a.table[0, 1] = a.pages
    a.table[2, 0] = -7
    a.call(Bn, 1, sel)
    assert int(a.status) == 0x4
    a.status.zero_()
    assert torch.isfinite(a.out).all()
    assert torch.equal(a.out[a.cu[1]:a.cu[2]], before[a.cu[1]:a.cu[2]])
    kept = (torch.arange(200, device="cuda") // 64 != 1).nonzero()[:, 0].int()
    if not k:
        b = Att(torch, [200, 100, 150, 64], [nq] * 4, Hq, 1, 128, 64, torch.bfloat16)
        row = kept.repeat(b.T, 1).contiguous()
        o, _, otol, _ = ref.attention(b.q, b.pool, 64, 1, good, b.lens, b.cu, 1, b.scale, row)
        n = a.cu[1]
        assert ((a.out[:n].double() - o[:n]).abs() <= otol[:n]).all()
    # lengths that break their bounds: the sequence's rows stay as they were
    a.table = good
    for lens, cu in (([201, 100, 150, 64], a.cu), ([-1, 100, 150, 64], a.cu)):
        a.out.fill_(77)
        a.lse.fill_(77)
        a.dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        a.call(Bn, 1, sel)
        assert int(a.status) == 0x10
        a.status.zero_()
        assert (a.out[:nq] == 77).all() and (a.lse[:nq] == 77).all()
        assert torch.equal(a.out[nq:], before[nq:])
    a.dev_lens = torch.tensor(a.lens, dtype=torch.int32, device="cuda")
    a.dev_cu = torch.tensor([0, nq, 2 * nq, 3 * nq, 4 * nq + 9], dtype=torch.int32, device="cuda")
    a.out.fill_(77)
    a.call(Bn, 1, sel)
    assert int(a.status) == 0x10
    assert torch.equal(a.out[:3 * nq], before[:3 * nq]) and (a.out[3 * nq:] == 77).all()


@pytest.mark.parametrize("Hq,k", [(8, 0), (64, 0), (8, 9), (64, 9)])
def test_more_queries_than_the_bound(torch, Bn, Hq, k):
    """A sequence with more queries than max_q_len is left alone; the others are not."""
    a = Att(torch, [50, 60, 70], [2, 9, 1], Hq, 1, 64, 64, torch.float16, pad=1)
    sel = lists(torch, a, 1, k) if k else None
    Bn.idx_attn_paged(a.q, a.pool, a.pages, 64, a.pool.stride(0), 1, a.table, a.dev_lens, a.dev_cu, 1, 4, 70, a.scale,
                      a.out, lse=a.lse, sel_idx=sel, dev_status=a.status)
    assert int(a.status) == 0x10 and (a.out[2:11] == 77).all() and (a.lse[2:11] == 77).all()
    o, _, otol, _ = ref.attention(a.q, a.pool, 64, 1, a.table, a.lens, a.cu, 1, a.scale, sel)
    keep = [0, 1, 11]
    assert ((a.out.double() - o).abs()[keep] <= otol[keep]).all()


@pytest.mark.parametrize("Hq,k", [(8, 0), (64, 0), (8, 5), (64, 5)])
def test_no_keys_at_all(torch, Bn, Hq, k):
    """Every sequence empty, with a page table of no columns: zeros and -inf, also with splits to spare."""
    a = Att(torch, [0, 0], [3, 1], Hq, 1, 128, 64, torch.bfloat16, width_extra=0, pad=2)
    sel = torch.full((a.T, k), 3, dtype=torch.int32, device="cuda") if k else None
    for ws in (None, torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")):
        a.out.fill_(77)
        a.call(Bn, 1, sel, ws)
        a.check(1, sel)


def test_one_key_among_splits_that_have_none(torch, Bn):
    """max_seq_len_k far above the lengths: most splits are empty and their parts of the workspace
    hold what was there before."""
    for Hq in (8, 64):
        a = Att(torch, [1, 130], [1, 1], Hq, 1, 128, 64, torch.bfloat16, width_extra=600)
        ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        Bn.idx_attn_paged(a.q, a.pool, a.pages, 64, a.pool.stride(0), 1, a.table, a.dev_lens, a.dev_cu, 1, 1, 38000, a.scale,
                          a.out, lse=a.lse, workspace=ws, dev_status=a.status)
        a.check(1)


def test_far_pages(torch, Bn):
    """Pages past 2^32 bytes of the pool, dense, selected, and with many rows."""
    stride, P, D = 1 << 28, 64, 128
    for Hq, nq, k in ((8, 1, 0), (64, 1, 0), (8, 1, 50), (64, 1, 50), (8, 40, 0)):
        a = Att(torch, [150, 90], [nq, nq], Hq, 1, D, P, torch.bfloat16)
        big = torch.zeros(17 + a.pages, stride, dtype=torch.uint8, device="cuda")
        big[17:, :a.pool.shape[1]] = a.pool
        sel = lists(torch, a, 1, k) if k else None
        a.call(Bn, 1, sel)
        first = a.out.clone()
        a.table = torch.where(a.table >= 0, a.table + 17, a.table)
        a.pool, a.pages = big, a.pages + 17
        a.out.fill_(77)
        a.call(Bn, 1, sel)
        assert torch.equal(first, a.out) and int(a.status) == 0
        del big, a


def test_streams_and_graphs(torch, Bn):
    """A side stream; a captured step replayed on new inputs; two graphs that share a workspace in
    turn."""
    a = Att(torch, [900, 333], [1, 1], 8, 2, 128, 64, torch.bfloat16)
    sel = lists(torch, a, 0, 64)
    ws = a.workspace(Bn)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.call(Bn, 0, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    a.check(0)
    dense, listed = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    o2, l2 = torch.zeros_like(a.out), torch.zeros_like(a.lse)
    keep = a.out, a.lse
    with torch.cuda.graph(dense):
        a.call(Bn, 0, ws=ws)
    a.out, a.lse = o2, l2
    with torch.cuda.graph(listed):
        a.call(Bn, 0, sel, ws)
    for seed in (1, 2):
        a.q.copy_(torch.randn(a.q.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        dense.replay()
        listed.replay()
        dense.replay()
        a.out, a.lse = keep
        a.check(0)
        a.out, a.lse = o2, l2
        a.check(0, sel)


def test_two_streams_at_once(torch, Bn):
    """Metadata, stores and attention of two batches on two streams at the same time, a workspace each:
    the bits of one after the other."""
    def batch(seed):
        a = Att(torch, [3000 + seed, 700], [1, 1], 64 if seed else 8, 1, 128, 64, torch.bfloat16, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        m = dict(ctx=torch.tensor([100 + seed, 63], **i32), new=torch.tensor([5, 9], **i32),
                 table=torch.full((2, 4), 1, **i32), free=torch.arange(2, 30, **i32), span=torch.tensor([0, 20], **i32),
                 cu=torch.zeros(3, **i32), lens=torch.zeros(2, **i32), pos=torch.zeros(16, **i32),
                 slots=torch.zeros(16, dtype=torch.int64, device="cuda"), nxt=torch.zeros(1, **i32))
        kv = torch.randn(16, 2, 1, 128, device="cuda", generator=g).bfloat16()
        pool = torch.zeros(40, 2 * 64 * 128 + 16, dtype=torch.uint8, device="cuda")
        return a, m, kv, pool, a.workspace(Bn)

    def run(b):
        a, m, kv, pool, ws = b
        for _ in range(20):
            Bn.idx_step_meta(m["ctx"], m["new"], m["table"], 64, 256, m["free"], m["span"], 40, m["cu"], m["lens"], m["pos"],
                             m["slots"], m["nxt"])
            Bn.idx_kv_store(kv[:, 0], kv[:, 1], m["slots"], pool, 40, 64, pool.stride(0))
            a.call(Bn, 0, ws=ws)

    both = [batch(0), batch(1)]
    want = []
    for b in both:
        run(b)
        torch.cuda.synchronize()
        want.append([x.clone() for x in (b[0].out, b[0].lse, b[1]["slots"], b[3])])
        for x in (b[0].out, b[0].lse, b[1]["slots"], b[3]):
            x.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, b in zip(streams, both):
        with torch.cuda.stream(s):
            run(b)
    torch.cuda.synchronize()
    for b, w in zip(both, want):
        for x, y in zip((b[0].out, b[0].lse, b[1]["slots"], b[3]), w):
            assert torch.equal(x, y)


def test_step_of_all_together(torch, Bn):
    """Three decode steps of a sparse layer as a program runs them: metadata from the lengths, the
    indexer's K store and Q quant, its scores and top-k, the KV store, and the attention over the
    selected keys; against the 64-bit form with the same keys."""
    from sparse_attention_indexer_mqa_gb300 import workloads as W
    B, P, H, D, Hq, Hkv, k, steps = 5, 64, 8, 128, 16, 1, 48, 3
    dev = dict(device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)
    start = [0, 63, 64, 100, 190]
    longest, pages = 256, 32
    table = torch.full((B, 4), -1, **i32)
    free = torch.randperm(pages, device="cuda", generator=g).int()
    span = torch.tensor([0, pages], **i32)
    cos_sin = torch.from_numpy(W.rope_table(longest)).cuda()
    ipool = torch.zeros(pages, W.page_bytes(W.MXFP4, P), dtype=torch.uint8, **dev)
    kpool = torch.full((pages, Hkv * (2 * P * D + 16)), 0x7F, dtype=torch.uint8, **dev)
    cpu_pool = kpool.cpu()
    status = torch.zeros(1, **i32)
    ctx = torch.zeros(B, **i32)
    for step in range(steps + 1):
        new = torch.tensor(start if step == 0 else [1] * B, **i32)
        T = int(new.sum()) + 2  # padded rows
        cu, lens, pos = torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(T, **i32)
        slots, nxt = torch.zeros(T, dtype=torch.int64, **dev), torch.zeros(1, **i32)
        ik = torch.randn(T, 128, generator=g, **dev).bfloat16()
        iq = torch.randn(T, H, 128, generator=g, **dev).bfloat16()
        w_in = torch.randn(T, H, generator=g, **dev)
        kv = torch.randn(T, 2, Hkv, D, generator=g, **dev).bfloat16()
        q = torch.randn(T, Hq, D, generator=g, **dev).bfloat16()
        codes, scales = torch.zeros(T, H, 64, dtype=torch.uint8, **dev), torch.zeros(T, 512, dtype=torch.uint8, **dev)
        w, logits = torch.zeros(T, H, **dev), torch.zeros(T, longest, **dev)
        top, out, lse = torch.zeros(T, k, **i32), torch.full((T, Hq, D), 77.0, **dev).bfloat16(), torch.full((T, Hq), 77.0, **dev)
        mq = int(new.max())
        Bn.idx_step_meta(ctx, new, table, P, longest, free, span, pages, cu, lens, pos, slots, nxt, dev_status=status)
        Bn.idx_qk_prep(ik.view(torch.int16), slots, pos, Bn.IDX_ROPE_NEOX, 1, ipool, pages, P, ipool.stride(0),
                       iq.view(torch.int16), pos, Bn.IDX_ROPE_NEOX, w_in, 1.0, 1.0, codes, scales, w, cos_sin,
                       Bn.IDX_MXFP4, dev_status=status)
        Bn.idx_mqa_logits_paged(codes, scales, w, Bn.IDX_MXFP4, ipool, pages, P, ipool.stride(0), table, lens, cu, 1,
                                mq, longest, logits, dev_status=status)
        Bn.idx_topk(logits, lens, cu, 1, longest, k, top, dev_status=status)
        Bn.idx_kv_store(kv[:, 0], kv[:, 1], slots, kpool, pages, P, kpool.stride(0), dev_status=status)
        Bn.idx_attn_paged(q, kpool, pages, P, kpool.stride(0), Hkv, table, lens, cu, 1, mq, longest, D ** -0.5, out,
                          lse=lse, sel_idx=top, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        cpu_pool = ref.store(cpu_pool, kv[:, 0].cpu(), kv[:, 1].cpu(), slots.cpu(), P)
        assert torch.equal(kpool.cpu(), cpu_pool)
        n = lens.tolist()
        assert n == [x + min(step, 1) * step for x in start] if step else n == start
        c = cu.tolist()
        for b in range(B):  # what the top-k lists is visible, distinct and complete
            for i, v in enumerate(ref.visible(n[b], c[b + 1] - c[b], 1)):
                row = [x for x in top[c[b] + i].tolist() if x >= 0]
                assert len(set(row)) == len(row) == min(v, k) and all(x < v for x in row)
        o, l, otol, ltol = ref.attention(q, kpool, P, Hkv, table, n, c, 1, D ** -0.5, top)
        own = ~torch.isnan(l)
        assert ((out.double() - o).abs()[own] <= otol[own]).all() and (out[~own] == 77).all()
        full = own & (l > -math.inf)
        assert ((lse.double() - l).abs()[full] <= ltol[full]).all()
        ctx = lens.clone()
        span = torch.cat([nxt, span[1:]])
