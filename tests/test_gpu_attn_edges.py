"""Calls of the step metadata and the paged attention at the borders of what include/idx.h allows, on the GPU."""
import math
import threading
import time

import pytest

import attn_ref as ref
from test_gpu_attn import Att, Bn, empty_pool, make_rows, run_meta, run_store, torch  # noqa: F401  (fixtures, inputs)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ NaN codes

def plant(a, b, pos, side, dim, head=0):
    """A NaN code in the cache: sequence b, key pos, K (0) or V (1)."""
    codes, _ = ref.kv_views(a.pool, a.Hkv, a.P, a.D)
    codes[int(a.table[b, pos // a.P]), head, pos % a.P, side, dim] = 0x7F if dim % 2 else 0xFF


NAN_SHAPES = [(8, 1, 2, 128, 64, "bfloat16"), (4, 2, 7, 64, 64, "float16"), (16, 1, 2, 64, 128, "bfloat16"),
              (64, 1, 2, 128, 128, "float16"), (24, 2, 3, 64, 64, "bfloat16"), (8, 1, 70, 128, 64, "bfloat16"),
              (1, 1, 150, 64, 128, "float16"), (3, 1, 300, 128, 128, "bfloat16")]


@pytest.mark.parametrize("Hq,Hkv,nq,D,P,dt", NAN_SHAPES)
@pytest.mark.parametrize("split", [False, True])
def test_nan_codes_stay_with_the_rows_that_see_them(torch, Bn, Hq, Hkv, nq, D, P, dt, split):
    """Slots that hold NaN codes before they are stored to: a causal row that does not see such a key has the
    result of the cache without it, though the row behind it in the same tile sees it."""
    extra = 9000 if split else 0
    a = Att(torch, [nq + 61 + extra, nq, nq + 127 + extra, nq + 3], [nq] * 4, Hq, Hkv, D, P, getattr(torch, dt), nq + D)
    n = a.lens
    clean, cl = torch.zeros_like(a.out), torch.zeros_like(a.lse)
    a.call(Bn, 1, ws=a.workspace(Bn) if split else None)
    clean.copy_(a.out), cl.copy_(a.lse)
    marks = [(0, n[0] - 1, 1, 5), (1, n[1] - 1, 1, D - 1), (1, n[1] - nq // 2, 1, 0), (2, n[2] - 1, 0, 7), (3, 1, 1, 33),
             (3, n[3] - 1, 1, 2)]
    for m in marks:
        plant(a, *m, head=Hkv - 1)
    a.call(Bn, 1, ws=a.workspace(Bn) if split else None)
    G = Hq // Hkv
    hit = torch.zeros(a.T, Hq, D, dtype=torch.bool, device="cuda")   # NaN by the definition
    seen = torch.zeros(a.T, Hq, dtype=torch.bool, device="cuda")     # a NaN code is among the row's keys
    hit_lse = torch.zeros(a.T, Hq, dtype=torch.bool, device="cuda")
    for b, pos, side, dim in marks:
        for i, v in enumerate(ref.visible(n[b], nq, 1)):
            if v > pos:
                hs = slice((Hkv - 1) * G, Hkv * G)
                seen[a.cu[b] + i, hs] = True
                if side:
                    hit[a.cu[b] + i, hs, dim] = True
                else:
                    hit[a.cu[b] + i, hs] = hit_lse[a.cu[b] + i, hs] = True
    assert int(a.status) == 0
    assert torch.equal(a.out[~seen], clean[~seen]) and torch.equal(a.lse[~hit_lse], cl[~hit_lse])
    assert torch.isnan(a.out[hit]).all() and torch.isnan(a.lse[hit_lse]).all()
    # the other dims of a row that sees a NaN code of V: NaN, or what they are without it
    left = seen[..., None] & ~hit & ~torch.isnan(a.out)
    assert torch.equal(a.out[left], clean[left])


@pytest.mark.parametrize("Hq", [8, 64])
def test_nan_codes_behind_every_row(torch, Bn, Hq):
    """Not causal, every row sees the same keys: a NaN code of V is NaN in its dim alone."""
    a = Att(torch, [70, 200], [2, 2], Hq, 1, 128, 64, torch.bfloat16)
    a.call(Bn, 0)
    clean = a.out.clone()
    plant(a, 0, 69, 1, 9)
    plant(a, 1, 3, 1, 10)
    a.call(Bn, 0)
    want = clean.clone()
    want[:2, :, 9] = math.nan
    want[2:, :, 10] = math.nan
    assert torch.equal(a.out.isnan(), want.isnan())
    assert torch.equal(a.out.nan_to_num(), want.nan_to_num())


# ------------------------------------------------------------------------------ rows without keys

@pytest.mark.parametrize("Hq,nq", [(8, 1), (64, 1), (64, 3), (17, 1)])
@pytest.mark.parametrize("k", [5, 700, 1500])
@pytest.mark.parametrize("split", [False, True])
def test_non_finite_query_without_keys(torch, Bn, Hq, nq, k, split):
    """A row whose list holds nothing that counts has out 0 and lse -inf whatever its query holds; one key makes it
    NaN."""
    a = Att(torch, [100, 90, 80], [nq] * 3, Hq, 1, 128, 64, torch.bfloat16)
    sel = torch.full((a.T, k), -1, dtype=torch.int32, device="cuda")
    sel[:, 1::2] = 100
    sel[2 * nq:, k - 1] = 0
    for value in (math.nan, math.inf):
        a.q[:, ::2, 3] = value
        a.out.fill_(77)
        a.lse.fill_(77)
        a.call(Bn, 1, sel, a.workspace(Bn, k) if split else None)
        assert int(a.status) == 0
        assert (a.out[:2 * nq] == 0).all() and (a.lse[:2 * nq] == -math.inf).all()
        assert a.out[2 * nq:, ::2].isnan().all() and a.lse[2 * nq:, ::2].isnan().all()
        assert a.out[2 * nq:, 1::2].isfinite().all() and a.lse[2 * nq:, 1::2].isfinite().all()


@pytest.mark.parametrize("Hq,nq", [(8, 1), (64, 1), (4, 40)])
def test_non_finite_query_on_pages_outside_the_pool(torch, Bn, Hq, nq):
    a = Att(torch, [130, 90], [nq, nq], Hq, 1, 64, 64, torch.float16)
    a.table[0] = a.pages
    a.q[:, 1] = math.inf
    a.call(Bn, 1)
    assert int(a.status) == Bn.IDX_STATUS_BAD_PAGE
    assert (a.out[:nq] == 0).all() and (a.lse[:nq] == -math.inf).all()
    assert a.out[nq:, 1].isnan().all() and a.out[nq:, 0].isfinite().all()


# ------------------------------------------------------------------------------ long lists

def graded(torch, a):
    """K and V scales of a's blocks over 17 exponents, the same in every head; the exponents by position."""
    _, scales = ref.kv_views(a.pool, a.Hkv, a.P, a.D)
    grade = []
    for b, n in enumerate(a.lens):
        block = torch.arange(-(-n // 16), device="cuda")
        g = block % 17
        page = a.table[b, block * 16 // a.P].long()
        e = torch.stack([104 + g, 122 - g], -1).to(torch.uint8)
        scales[page, :, block * 16 % a.P // 16] = e[:, None]
        grade.append(g.repeat_interleave(16)[:n].cpu())
    return grade


def stepped(torch, a, k, seed):
    """Lists whose steps of 128 entries are of unlike kinds: scales all alike, 2^15 apart (the most that is folded
    into the operands), 2^16 apart, with one entry that does not count, of such entries alone, random."""
    grade = graded(torch, a)
    g = torch.Generator().manual_seed(seed)
    sel = torch.full((a.T, k), -1, dtype=torch.int32)

    def some(ids, count):
        return ids[torch.randint(len(ids), (count,), generator=g)]
    for b, n in enumerate(a.lens):
        at = torch.arange(n)
        kinds = [lambda c: some(at[grade[b] == 4], c), lambda c: some(at[grade[b] <= 15], c),
                 lambda c: some(at, c), lambda c: some(at[grade[b] <= 1], c),
                 lambda c: torch.full((c,), n), lambda c: some(at[grade[b] > 0], c)]
        for t in range(a.cu[b], a.cu[b + 1]):
            for i, start in enumerate(range(0, k, 128)):
                count = min(128, k - start)
                part = kinds[(i + t) % len(kinds)](count)
                if (i + t) % len(kinds) == 3:
                    part[int(torch.randint(count, (1,), generator=g))] = -1
                sel[t, start:start + count] = part.int()
    return sel.cuda()


@pytest.mark.parametrize("Hq,Hkv,D,dt", [(8, 1, 128, "bfloat16"), (16, 1, 64, "float16"), (64, 1, 128, "float16"),
                                         (130, 1, 64, "bfloat16"), (40, 2, 128, "bfloat16"), (34, 2, 128, "float16")])
@pytest.mark.parametrize("k", [1024, 2048, 1500])
@pytest.mark.parametrize("split", [False, True])
def test_long_lists(torch, Bn, Hq, Hkv, D, dt, k, split):
    """Lists of many steps, split and joined or whole, folded steps and others in one row; full lists of distinct keys
    and lists of steps of unlike kinds."""
    a = Att(torch, [5000, 2100, 3333], [1, 2, 1], Hq, Hkv, D, 64, getattr(torch, dt), k + Hq)
    g = torch.Generator().manual_seed(k)
    full = torch.stack([torch.randperm(2100, generator=g)[:k] for _ in range(a.T)]).int()
    full = torch.nn.functional.pad(full, (0, k - full.shape[1]), value=-1).cuda()
    ws = a.workspace(Bn, k) if split else None
    if split:
        assert ws.numel() > 256
    a.call(Bn, 0, full, ws)
    a.check(0, full)
    sel = stepped(torch, a, k, k + Hq)
    a.scale = 2.0 ** -4 / D
    a.out.fill_(77), a.lse.fill_(77)
    a.call(Bn, 0, sel, ws)
    a.check(0, sel)


# ------------------------------------------------------------------------------ ends of the ranges

@pytest.mark.parametrize("Hq,nq,k", [(8, 1, 0), (64, 1, 0), (8, 3, 0), (8, 40, 0), (8, 1, 300), (64, 1, 300), (17, 2, 129)])
@pytest.mark.parametrize("split", [False, True])
def test_scales_at_the_ends_of_their_range(torch, Bn, Hq, nq, k, split):
    """Scale exponents -32 and 48 side by side, V's in every row, K's with logits that stay small; bytes that the store
    does not write are read as the nearest that it does."""
    a = Att(torch, [2100, 260], [nq, nq], Hq, 1, 128, 64, torch.bfloat16, k + Hq)
    _, scales = ref.kv_views(a.pool, 1, 64, 128)
    g = torch.Generator().manual_seed(1)
    ends = torch.tensor([95, 175, 121], dtype=torch.uint8)
    scales[..., 1] = ends[torch.randint(3, scales.shape[:-1], generator=g)].cuda()
    scales[..., 0] = torch.tensor([95, 100], dtype=torch.uint8)[torch.randint(2, scales.shape[:-1], generator=g)].cuda()
    a.scale = 2.0 ** 16
    sel = None
    if k:
        sel = torch.stack([torch.randperm(260 - nq, generator=g)[:k] if k < 250 else torch.randint(260 - nq, (k,), generator=g)
                           for _ in range(a.T)]).int().cuda()
    ws = a.workspace(Bn, k) if split else None
    a.call(Bn, 1, sel, ws)
    a.check(1, sel)
    kept = a.out.clone(), a.lse.clone()
    scales[..., 1] = torch.where(scales[..., 1] == 95, 0, torch.where(scales[..., 1] == 175, 255, scales[..., 1]))
    scales[..., 0] = torch.where(scales[..., 0] == 95, 7, scales[..., 0])
    a.call(Bn, 1, sel, ws)
    assert torch.equal(a.out, kept[0]) and torch.equal(a.lse, kept[1])


@pytest.mark.parametrize("Hq,nq", [(4, 1), (64, 1), (4, 70)])
def test_small_and_large_fp16_queries(torch, Bn, Hq, nq):
    """Rows of q in fp16's subnormal range, zeros, and rows near its largest value."""
    a = Att(torch, [200], [nq], Hq, 1, 64, 64, torch.float16)
    a.scale = 2.0 ** -10
    for i, f in enumerate([0.0, 2.0 ** -20, 2.0 ** -14, 2.0 ** 13]):
        a.q[:, i] = (a.q[:, i].float().clamp(-4, 4) * f).half()
    a.call(Bn, 1)
    a.check(1)


# ------------------------------------------------------------------------------ batches of unlike requests

@pytest.mark.parametrize("Hq,Hkv,D,dt", [(8, 1, 128, "bfloat16"), (16, 2, 64, "float16"), (64, 1, 128, "float16"),
                                         (1, 1, 64, "bfloat16"), (32, 8, 128, "bfloat16")])
@pytest.mark.parametrize("split", [False, True])
def test_decodes_beside_a_chunk(torch, Bn, Hq, Hkv, D, dt, split):
    """Single tokens on caches of unlike lengths, a chunk of a prompt, requests without tokens, in one call."""
    nq = [1] * 20 + [0, 170, 0] + [1] * 13 + [3]
    lens = [1 + 97 * i for i in range(20)] + [40, 1234, 0] + [2000 + 31 * i for i in range(13)] + [3]
    a = Att(torch, lens, nq, Hq, Hkv, D, 128, getattr(torch, dt), Hq, pad=5)
    a.call(Bn, 1, ws=a.workspace(Bn) if split else None)
    a.check(1)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (40, 1), (6, 3)])
def test_many_short_requests(torch, Bn, Hq, Hkv):
    a = Att(torch, [1 + (i * 37) % 150 for i in range(500)], [1] * 500, Hq, Hkv, 64, 64, torch.float16, Hq, pad=1)
    a.call(Bn, 1, ws=a.workspace(Bn))
    a.check(1)


# ------------------------------------------------------------------------------ stores of many rows

@pytest.mark.parametrize("H,D,P,dt", [(1, 64, 64, "float16"), (5, 128, 128, "bfloat16")])
@pytest.mark.parametrize("case", ["prompt", "tokens", "gaps", "flagged"])
def test_store_many_rows(torch, Bn, H, D, P, dt, case):
    """1024 rows and more, of which a CTA looks at 16: runs that cross its rows, single tokens of many requests, rows
    that are skipped or refused at its borders."""
    n, status = 1300, 0
    perm = torch.randperm(1400, generator=torch.Generator().manual_seed(3)).tolist()
    if case == "prompt":      # two prompts that begin inside a block
        slots = list(range(5, 705))
        first = (705 // P + 1) * P
        slots += [first + 9 + i for i in range(n - 700)]
        pages = slots[-1] // P + 1
    elif case == "tokens":    # one token of each of 1300 requests, at any offset of a block of its own
        slots = [16 * b + b % 16 for b in perm[:n]]
        pages = 1400 * 16 // P + 1
    else:
        slots = list(range(3, 3 + n))
        pages = n // P + 2
        if case == "gaps":    # whole blocks left out, among them some at the borders of 16 rows
            slots = [-1 if s // 16 % 5 == 2 else s for s in slots]
        else:
            status = 1
            for r in (16, 32, 47, 255, 256, 1299):   # a slot twice: it and the block's rows behind it are skipped
                slots[r] = slots[r - 1]
            slots[600] = pages * P                   # past the pool
            for r in range(601, 603 + 16):           # the rest of that row's block: apart from its first rows
                if slots[r] // 16 == slots[599] // 16:
                    slots[r] = -1
    pool = empty_pool(torch, pages, H, D, P, 5)
    run_store(torch, Bn, pool, make_rows(torch, n, H, D, getattr(torch, dt), 6), slots, P, status)


# ------------------------------------------------------------------------------ step metadata

def decode_step(torch, Bn, B, T_extra=0, seed=0):
    """The inputs and outputs of a decode step of B requests, its call, and the slots it has to give."""
    P = 64
    g = torch.Generator().manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = torch.randint(0, 2 * P, (B,), generator=g)
    table = torch.arange(4 * B, **i32).reshape(B, 4).contiguous()
    free = torch.arange(4 * B, 6 * B, **i32)
    T = B + T_extra
    t = dict(ctx=ctx.to(**i32), new=torch.ones(B, **i32), table=table, free=free, span=torch.tensor([0, 2 * B], **i32),
             cu=torch.zeros(B + 1, **i32), lens=torch.zeros(B, **i32), pos=torch.zeros(T, **i32),
             slots=torch.zeros(T, dtype=torch.int64, device="cuda"), nxt=torch.zeros(1, **i32))
    fresh = ctx % P == 0
    order = torch.cumsum(fresh.long(), 0) - 1
    page = torch.where(fresh, 4 * B + order, 4 * torch.arange(B) + ctx // P)
    want = torch.cat([page * P + ctx % P, torch.full((T_extra,), -1)])

    def call(**kw):
        Bn.idx_step_meta(t["ctx"], t["new"], t["table"], P, 4 * P, t["free"], t["span"], 6 * B, t["cu"], t["lens"],
                         t["pos"], t["slots"], t["nxt"], **kw)
    return t, call, want


def test_meta_of_unlike_batches_from_threads(torch, Bn):
    """Host threads whose batches need unlike amounts of shared memory."""
    errors, made = [], [decode_step(torch, Bn, B, 3, B) for B in (16384, 6200, 9000)]
    torch.cuda.synchronize()
    gate = threading.Barrier(len(made))

    def work(t, call, want):
        try:
            stream = torch.cuda.Stream()
            gate.wait()
            for _ in range(1500):
                call(stream=stream)
            stream.synchronize()
            assert torch.equal(t["slots"].cpu(), want)
        except Exception as e:  # seen by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=m) for m in made]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors, errors


@pytest.mark.parametrize("new,P", [([60000], 64), ([1, 0, 33333, 5], 128), ([0, 1, 20000, 20000], 64)])
def test_meta_of_long_prompts(torch, Bn, new, P):
    """Hundreds of pages to a request, on shuffled pages, beside single tokens."""
    ctx = [(7 * i) % 130 for i in range(len(new))]
    longest = max(x + y for x, y in zip(ctx, new))
    need = sum(-(-(x + y) // P) - -(-x // P) for x, y in zip(ctx, new))
    free = torch.randperm(need + 50, generator=torch.Generator().manual_seed(1)).tolist()
    run_meta(torch, Bn, ctx, new, P, longest, free, [2, 2 + need], need + 50, sum(new) + 3, -(-longest // P) + 1, 1, 0)


@pytest.mark.parametrize("between", ["nothing", "capture", "refused", "names"])
def test_lengths_reach_the_next_call_whatever_lies_between(torch, Bn, between):
    """The top-k reads lengths before it waits for the kernel in front of it. Eager metadata and top-k with a
    capture on the same stream between them, a refused call, or another name of the same stream."""
    t, call, _ = decode_step(torch, Bn, 512)
    L, k = 256, 4
    logits = torch.arange(L, device="cuda").float().repeat(512, 1).contiguous()
    got = [torch.zeros(512, k, dtype=torch.int32, device="cuda") for _ in range(40)]
    ctx = torch.randint(4, 200, (len(got), 512), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    first, second = (0, 1) if between == "names" else (side, side)  # 1: cudaStreamLegacy
    torch.cuda.synchronize()
    graphs = []
    for i, out in enumerate(got):
        with torch.cuda.stream(torch.cuda.default_stream() if between == "names" else side):
            t["ctx"].copy_(ctx[i])
            call(stream=first)
            if between == "capture":
                graphs.append(torch.cuda.CUDAGraph())
                graphs[-1].capture_begin()
                Bn.idx_topk(logits, t["lens"], t["cu"], 0, L, k, torch.zeros_like(out), stream=side)
                graphs[-1].capture_end()
            elif between == "refused":
                with pytest.raises(Bn.IdxError):
                    Bn.idx_topk(logits, t["lens"], t["cu"], 0, L, 0, out, stream=side)
            Bn.idx_topk(logits, t["lens"], t["cu"], 0, L, k, out, stream=second)
    torch.cuda.synchronize()
    n = ctx.long() + 1
    want = torch.stack([n - 3, n - 2, n - 1, n - 4], -1).int()  # above the k-th in index order, then the k-th
    wrong = (torch.stack(got) != want).any(-1).nonzero()
    assert len(wrong) == 0, (len(wrong), [(n[i, b].item(), got[i][b].tolist()) for i, b in wrong[:4].tolist()])


def test_two_streams_in_turns(torch, Bn):
    """Metadata, store and attention of two batches on two streams, call by call in turn: the bits of one
    after the other."""
    P, H, D = 64, 1, 128

    def batch(seed):
        B = 300 + 100 * seed
        t, call, want = decode_step(torch, Bn, B, 5, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        kv = torch.randn(B + 5, 2, H, D, device="cuda", generator=g).bfloat16()
        q = torch.randn(B + 5, 16 + 48 * seed, D, device="cuda", generator=g).bfloat16()
        pool = torch.zeros(6 * B, 2 * P * D + 16, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)

        def attend(stream):
            Bn.idx_attn_paged(q, pool, 6 * B, P, pool.stride(0), H, t["table"], t["lens"], t["cu"], 1, 1, 4 * P, 0.1, out,
                              stream=stream)
        steps = [lambda s: call(stream=s),
                 lambda s: Bn.idx_kv_store(kv[:, 0], kv[:, 1], t["slots"], pool, 6 * B, P, pool.stride(0), stream=s),
                 attend, lambda s: (t["ctx"].copy_(t["lens"]), t["span"][:1].copy_(t["nxt"]))]
        ctx = t["ctx"].clone()

        def reset():
            t["ctx"].copy_(ctx)
            t["span"][:1].zero_()
            t["table"].copy_(torch.arange(4 * B, dtype=torch.int32, device="cuda").reshape(B, 4))
            pool.zero_()
            out.zero_()
        return steps, reset, (out, pool, t["slots"], t["lens"], t["table"]), want

    both = [batch(0), batch(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for (steps, reset, outs, want), s in zip(both, streams):
        with torch.cuda.stream(s):
            reset()
            steps[0](s)
            assert torch.equal(outs[2].cpu(), want)
            reset()
            for _ in range(30):
                for step in steps:
                    step(s)
            alone.append([x.clone() for x in outs])
            reset()
    torch.cuda.synchronize()
    for _ in range(30):
        for i in range(4):
            for (steps, _, _, _), s in zip(both, streams):
                with torch.cuda.stream(s):
                    steps[i](s)
    torch.cuda.synchronize()
    for (_, _, outs, _), want in zip(both, alone):
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("nq,Hq,keys", [(2000, 8, 2000), (1, 8, 30000), (1, 64, 30000), (40, 1, 9000), (1, 16, 500)])
@pytest.mark.parametrize("split", [False, True])
def test_output_as_the_next_calls_query(torch, Bn, nq, Hq, keys, split):
    """The Q quantisation reads q before it waits for the kernel in front of it: here the attention's output."""
    a = Att(torch, [keys, keys - 7], [nq, nq], Hq, 1, 128, 128, torch.bfloat16)
    ws = a.workspace(Bn) if split else None
    w = torch.ones(a.T, Hq, device="cuda")
    outs = [(torch.zeros(a.T, Hq + -Hq % 8, 64, dtype=torch.uint8, device="cuda"),
             torch.zeros(a.T, 512, dtype=torch.uint8, device="cuda"), torch.zeros_like(w)) for _ in range(8)]
    other = torch.randn(a.q.shape, device="cuda").bfloat16()
    qs = [a.q, other]

    def quant(o):
        Bn.idx_q_quant(a.out.view(torch.int16), None, None, Bn.IDX_ROPE_NONE, w, 1.0, 1.0, Bn.IDX_MXFP4, *o)
    want = []
    for i in range(2):
        a.q = qs[i]
        a.call(Bn, 1, ws=ws)
        torch.cuda.synchronize()
        o = tuple(torch.zeros_like(x) for x in outs[0])
        quant(o)
        torch.cuda.synchronize()
        want.append(o)
    assert not torch.equal(want[0][0], want[1][0])
    for i, o in enumerate(outs):
        a.q = qs[i % 2]
        a.call(Bn, 1, ws=ws)
        quant(o)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert all(torch.equal(x, y) for x, y in zip(o, want[i % 2])), i


def test_attention_waits_give_up_in_time(torch, Bn):
    """Both wait helpers at the kernels' own limit of a second each, on a barrier that nothing completes; an attention
    call right after runs."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    Bn.idx_debug_wait_timeout(1000000, status)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert int(status) == Bn.IDX_STATUS_TIMEOUT
    assert 1.2 < took < 2.6  # 1 s by the clock, then 250000 tests of 1 to 4.1 us
    a = Att(torch, [200, 100], [3, 2], 64, 1, 128, 64, torch.bfloat16)
    a.call(Bn, 1)
    a.check(1)
