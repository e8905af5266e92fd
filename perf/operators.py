"""Performance cases of the serving operators around the indexer's cache and top-k.

Three operators, used together in a serving step:

* ``step_meta``  -- page tables, slot map, positions and lengths of a step, built on the GPU
  from the requests' lengths and a list of free pages;
* ``kv_store``   -- new K and V rows into the 8-bit paged cache (e4m3 codes, one power-of-two
  scale per 16 tokens, kv head and side);
* ``attention``  -- softmax attention over that cache, over every visible key or over the keys
  that the indexer's top-k lists.

``run`` computes an operator with elementary torch operations in 32 bits while ``own`` is false,
and by the library's entry points while it is true. Lengths are functions of the case alone;
values come from the seed.

Cache page, as both sides read it: kv head h of a page starts at h * (2*P*D + 16) bytes; token s
of the head has its D K codes at s*2*D and its D V codes right behind them; the scale bytes
(exponent + 127) of 16-token block i are at 2*P*D + 2*i (K) and 2*P*D + 2*i + 1 (V).
"""
import math

import torch

own = False

BLOCK = 16                 # tokens of a scale block
E_MIN, E_MAX = -32, 48     # range of a block's scale exponent
WORKSPACE = 64 << 20       # bytes a program keeps for the attention's partial results
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ cases

def listed():
    att = dict(op="attention", type="bf16", D=128, P=128, causal=1, k=0, pad=0, empty_every=0)
    return [
        # one decode step's bookkeeping: 64 requests, one new token each
        dict(name="meta_decode_64", op="step_meta", B=64, P=128, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=8191,
             pad=0, short=0),
        # a mixed step of many requests: decodes and prompt chunks, a padded token capacity
        dict(name="meta_mixed_512", op="step_meta", B=512, P=64, q_lo=0, q_hi=255, ctx_lo=0, ctx_hi=16000,
             pad=777, short=0),
        # a decode step's new K and V rows, 8 kv heads
        dict(name="store_decode_64", op="kv_store", type="bf16", B=64, Hkv=8, D=128, P=128, q_lo=1, q_hi=1,
             ctx_lo=0, ctx_hi=500, pad=0),
        # a prompt of 8192 tokens
        dict(name="store_prefill_8k", op="kv_store", type="bf16", B=1, Hkv=8, D=128, P=128, q_lo=8192,
             q_hi=8192, ctx_lo=0, ctx_hi=0, pad=0),
        # ragged chunks that begin and end inside a scale block
        dict(name="store_chunks_odd", op="kv_store", type="fp16", B=37, Hkv=2, D=64, P=64, q_lo=1, q_hi=200,
             ctx_lo=0, ctx_hi=333, pad=5),
        # one short request: latency alone
        dict(att, name="attn_decode_one", type="fp16", B=1, Hq=8, Hkv=1, q_lo=1, q_hi=1, ctx_lo=256,
             ctx_hi=256, causal=0),
        # a decode step of 64 requests with full caches
        dict(att, name="attn_decode_64", B=64, Hq=64, Hkv=8, q_lo=1, q_hi=1, ctx_lo=8191, ctx_hi=8191),
        # two long contexts: the key axis has to be split
        dict(att, name="attn_decode_long", B=2, Hq=32, Hkv=4, D=64, P=64, q_lo=1, q_hi=1, ctx_lo=131070,
             ctx_hi=131070, causal=0),
        # a causal prompt of 8192 tokens
        dict(att, name="attn_prefill_8k", B=1, Hq=32, Hkv=8, q_lo=8192, q_hi=8192, ctx_lo=0, ctx_hi=0),
        # ragged chunks on cached tokens, odd sizes, padded rows
        dict(att, name="attn_chunks_odd", type="fp16", B=8, Hq=12, Hkv=4, D=64, P=64, q_lo=3, q_hi=301,
             ctx_lo=0, ctx_hi=3001, pad=7),
        # decode over the indexer's 1024 keys per query, 64 heads that share the cache
        dict(att, name="attn_topk_decode_64", B=64, Hq=64, Hkv=1, q_lo=1, q_hi=1, ctx_lo=8191, ctx_hi=8191,
             k=1024),
        # a chunk of prompt over the indexer's keys
        dict(att, name="attn_topk_prefill", B=1, Hq=64, Hkv=1, q_lo=4096, q_hi=4096, ctx_lo=4096,
             ctx_hi=4096, k=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step_meta", "kv_store", "decode", "decode", "chunks", "topk", "topk"])
    if op == "step_meta":
        B = _log(rng, 1, 1024)
        q_hi = _log(rng, 1, max(1, 60000 // B))
        return dict(op=op, B=B, P=rng.choice([64, 128]), q_lo=rng.randint(0, 1), q_hi=q_hi, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 16000), pad=rng.choice([0, 3, _log(rng, 1, 500)]),
                    short=rng.choice([0, 0, 1]))
    if op == "kv_store":
        B, D = _log(rng, 1, 96), rng.choice([64, 128])
        return dict(op=op, type=rng.choice(["bf16", "fp16"]), B=B, Hkv=rng.choice([1, 2, 3, 4, 8]), D=D,
                    P=rng.choice([64, 128]), q_lo=rng.randint(0, 1), q_hi=_log(rng, 1, max(2, 6000 // B)),
                    ctx_lo=0, ctx_hi=_log(rng, 1, 700), pad=rng.choice([0, 0, 9]))
    c = dict(op="attention", type=rng.choice(["bf16", "fp16"]), D=rng.choice([64, 128]),
             P=rng.choice([64, 128]), causal=rng.choice([0, 1]), k=0, pad=rng.choice([0, 0, 5]),
             empty_every=rng.choice([0, 0, 3]))
    if op == "decode":
        B, Hkv = _log(rng, 1, 96), rng.choice([1, 2, 3, 4, 8])
        L = _log(rng, 1, max(2, min(120000, 3000000 // (B * Hkv))))
        c.update(B=B, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 7, 8, 16, 32]), q_lo=1,
                 q_hi=rng.choice([1, 1, 2, 4]), ctx_lo=rng.choice([0, L // 2, L]), ctx_hi=L)
    elif op == "chunks":
        B, Hkv = _log(rng, 1, 8), rng.choice([1, 2, 4, 8])
        c.update(B=B, Hkv=Hkv, Hq=Hkv * rng.choice([1, 3, 4, 8]), q_lo=rng.randint(0, 9),
                 q_hi=_log(rng, 17, 4096 // B), ctx_lo=0, ctx_hi=_log(rng, 1, 4000), causal=1)
    else:
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        q_hi = _log(rng, 1, max(1, 1000 // B))
        c.update(B=B, Hkv=Hkv, Hq=Hkv * rng.choice([4, 8, 16, 32, 64, 128] if Hkv == 1 else [2, 8, 16]), q_lo=1,
                 q_hi=q_hi, ctx_lo=0, ctx_hi=_log(rng, 16, 20000), k=rng.choice([32, 257, 1024, 2048]))
    return c


def _ragged(n, lo, hi, salt):
    """n lengths in [lo, hi], spread but fixed: a function of the arguments alone."""
    return [lo + ((i + salt) * 2654435761 % 4294967296 >> 7) % (hi - lo + 1) for i in range(n)]


def _lengths(c):
    ctx = _ragged(c["B"], c["ctx_lo"], c["ctx_hi"], 11)
    new = _ragged(c["B"], c["q_lo"], c["q_hi"], 5)
    if sum(new) == 0:
        new[0] = 1
    return ctx, new


def _seq_lens(c):
    """Keys of each sequence of an attention case; some have none although they have queries."""
    ctx, new = _lengths(c)
    e = c["empty_every"]
    return [0 if e and b % e == e - 1 else x + y for b, (x, y) in enumerate(zip(ctx, new))]


def _visible(c):
    """Keys that each query row sees, sequence after sequence."""
    _, new = _lengths(c)
    return [[min(max(n - q + i + 1, 0), n) if c["causal"] else n for i in range(q)]
            for n, q in zip(_seq_lens(c), new)]


def work(c):
    ctx, new = _lengths(c)
    if c["op"] == "step_meta":
        rows = sum(new) + c["pad"]
        pages = sum(-(-(x + y) // c["P"]) - -(-x // c["P"]) for x, y in zip(ctx, new))
        return {"bytes": 8 * c["B"] + 8 * (c["B"] + 1) + 8 * pages + 12 * rows, "flops": 0}
    if c["op"] == "kv_store":
        row = c["Hkv"] * c["D"]
        return {"bytes": sum(new) * (4 * row + 2 * row + 8) + 2 * c["Hkv"] * -(-sum(new) // BLOCK), "flops": 0}
    vis = _visible(c)
    seen = [min(v, c["k"]) if c["k"] else v for rows in vis for v in rows]
    key = c["Hkv"] * (2 * c["D"] + 0.125)
    if c["k"]:  # each cached key once at most, and each list
        keys = sum(min(max(rows, default=0), sum(min(v, c["k"]) for v in rows)) for rows in vis)
    else:
        keys = sum(max(rows, default=0) for rows in vis)
    rows = sum(new)
    return {"bytes": keys * key + rows * c["Hq"] * (4 * c["D"] + 4) + 4 * rows * c["k"],
            "flops": 4 * c["D"] * c["Hq"] * sum(seen)}


# ------------------------------------------------------------------------------ inputs

def _views(pool, c):
    """Codes [pages, Hkv, P, 2, D] and scale bytes [pages, Hkv, P/16, 2] of a pool, in place."""
    n, stride = pool.shape
    H, P, D = c["Hkv"], c["P"], c["D"]
    head = 2 * P * D + 16
    codes = pool.as_strided((n, H, P, 2, D), (stride, head, 2 * D, D, 1))
    scales = pool.as_strided((n, H, P // BLOCK, 2), (stride, head, 2, 1), 2 * P * D)
    return codes, scales


def _pages(lens, P, spare, gen, width):
    """A shuffled page table [B, width] (-1 where there is no page) and the pages left over."""
    need = [-(-n // P) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    start = need_t.cumsum(0) - need_t
    j = torch.arange(width, device="cuda")
    at = (start[:, None] + j).clamp(max=total - 1)
    table = torch.where(j < need_t[:, None], perm[at], -1).to(torch.int32)
    return table.contiguous(), perm[sum(need):].contiguous(), total


def _filled_pool(c, pages, gen):
    """A cache of `pages` pages with codes and scales as the store leaves them."""
    stride = c["Hkv"] * (2 * c["P"] * c["D"] + 16)
    pool = torch.zeros(pages, stride, dtype=torch.uint8, device="cuda")
    codes, scales = _views(pool, c)
    x = torch.empty(codes.shape, device="cuda", dtype=torch.bfloat16).normal_(0.0, 100.0, generator=gen)
    codes.copy_(x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    scales.copy_(torch.randint(119, 123, scales.shape, generator=gen, device="cuda", dtype=torch.uint8))
    return pool


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    ctx, new = _lengths(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    T = sum(new) + c["pad"]
    s = {"case": c, "T": T, "status": torch.zeros(1, **i32)}
    if c["op"] == "step_meta":
        P = c["P"]
        longest = max(x + y for x, y in zip(ctx, new))
        need = sum(-(-(x + y) // P) - -(-x // P) for x, y in zip(ctx, new))
        width = -(-longest // P) + 1
        table, free, pages = _pages(ctx, P, need + 40, gen, width)
        head = seed % 7
        end = head + need - (1 + need // 8 if c["short"] and need else 0)
        s.update(ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), table=table, free=free, pages=pages,
                 span=torch.tensor([head, end], **i32), longest=longest, cu=torch.zeros(c["B"] + 1, **i32),
                 lens=torch.zeros(c["B"], **i32), pos=torch.zeros(T, **i32),
                 slots=torch.zeros(T, dtype=torch.int64, device="cuda"), next=torch.zeros(1, **i32))
        return s
    lens = [x + y for x, y in zip(ctx, new)] if c["op"] == "kv_store" else _seq_lens(c)
    P, width = c["P"], max(1, -(-max(lens) // c["P"]))
    table, _, pages = _pages(lens, P, 2, gen, width)
    s["pool"] = _filled_pool(c, pages, gen)
    dt = TYPES[c["type"]]
    row_seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), torch.tensor(new, device="cuda"))
    cu = torch.tensor([0] + new, device="cuda").cumsum(0)
    i = torch.arange(sum(new), device="cuda") - cu[row_seq]
    if c["op"] == "kv_store":
        at = torch.tensor(ctx, device="cuda")[row_seq] + i
        slots = table[row_seq, at // P].to(torch.int64) * P + at % P
        s["slots"] = torch.cat([slots, slots.new_full((c["pad"],), -1)])
        kv = torch.randn(T, 2, c["Hkv"], c["D"], generator=gen, device="cuda")
        kv *= torch.rand(T, 2, c["Hkv"], 1, generator=gen, device="cuda") * 3 + 0.2  # rows of unlike size
        kv = kv.to(dt)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]  # as two halves of one projection's output
        return s
    # attention: slots past a sequence's length hold what earlier requests left, NaN codes here
    lens_t = torch.tensor(lens, **i32)
    codes, _ = _views(s["pool"], c)
    last = ((lens_t.long() - 1).clamp(min=0) // P).clamp(max=width - 1)
    page = table.gather(1, last[:, None])[:, 0].long().clamp(min=0)
    j = torch.arange(P, device="cuda")
    stale = (j >= (lens_t.long() - last * P)[:, None]) & (lens_t > 0)[:, None]
    codes[page] = torch.where(stale[:, None, :, None, None], 127, codes[page])
    s.update(table=table, lens=lens_t, cu=cu.to(torch.int32), max_q=max(new), max_k=max(lens),
             q=torch.randn(T, c["Hq"], c["D"], generator=gen, device="cuda").to(dt), scale=c["D"] ** -0.5,
             out=torch.zeros(T, c["Hq"], c["D"], dtype=dt, device="cuda"),
             lse=torch.zeros(T, c["Hq"], dtype=torch.float32, device="cuda"),
             workspace=torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda"), sel=None)
    if c["k"]:
        vis = torch.tensor([v for rows in _visible(c) for v in rows] + [0] * c["pad"], device="cuda")
        n = min(c["k"], s["max_k"])
        sel = torch.full((T, c["k"]), -1, **i32)
        rows = max(1, (1 << 28) // max(1, s["max_k"]))
        for at in range(0, T, rows):  # k distinct visible keys per row, by random keys
            v = vis[at:at + rows, None]
            r = torch.rand(v.shape[0], s["max_k"], generator=gen, device="cuda")
            r = torch.where(torch.arange(s["max_k"], device="cuda") < v, r, -1.0)
            top, idx = r.topk(n, dim=1)
            sel[at:at + rows, :n] = torch.where(top >= 0, idx, -1).to(torch.int32)
        s["sel"] = sel
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"step_meta": _own_meta, "kv_store": _own_store, "attention": _own_attention}[op](s)
    return {"step_meta": _plain_meta, "kv_store": _plain_store, "attention": _plain_attention}[op](s)


def _own_meta(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    idx.idx_step_meta(s["ctx"], s["new"], s["table"], s["case"]["P"], s["longest"], s["free"], s["span"], s["pages"],
                      s["cu"], s["lens"], s["pos"], s["slots"], s["next"], dev_status=s["status"])
    return {"table": s["table"], "cu": s["cu"], "lens": s["lens"], "pos": s["pos"], "slots": s["slots"],
            "next": s["next"]}


def _own_store(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    c = s["case"]
    idx.idx_kv_store(s["k"], s["v"], s["slots"], s["pool"], s["pool"].shape[0], c["P"], s["pool"].stride(0),
                     dev_status=s["status"])
    codes, scales = _views(s["pool"], c)
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}


def _own_attention(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    c = s["case"]
    idx.idx_attn_paged(s["q"], s["pool"], s["pool"].shape[0], c["P"], s["pool"].stride(0), c["Hkv"], s["table"],
                       s["lens"], s["cu"], c["causal"], s["max_q"], s["max_k"], s["scale"], s["out"], lse=s["lse"],
                       sel_idx=s["sel"], workspace=s["workspace"], dev_status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e in 32 bits for whole e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_meta(s):
    P, cap, longest = s["case"]["P"], s["T"], s["longest"]
    ctx, new = s["ctx"].long(), s["new"].long()
    n = new.clamp(min=0)
    end = n.cumsum(0)
    cu = torch.cat([end.new_zeros(1), end]).clamp(max=cap)
    ok = (ctx >= 0) & (new >= 0) & (ctx + new <= longest) & (end <= cap)
    old, full = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    need = torch.where(ok, full - old, 0)
    upto = need.cumsum(0)
    head, tail = s["span"].long().unbind()
    ok &= (need == 0) | (head + upto <= tail)
    first = head + upto - need
    j = torch.arange(s["table"].shape[1], device=ctx.device)
    fresh = ok[:, None] & (j >= old[:, None]) & (j < full[:, None])
    at = (first[:, None] + j - old[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    t = torch.arange(cap, device=ctx.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = b < ctx.numel()
    b = b.clamp(max=ctx.numel() - 1)
    live &= ok[b]
    pos = torch.where(live, ctx[b] + t - cu[b], 0)
    page = table[b, (pos // P).clamp(max=table.shape[1] - 1)].long()
    return {"table": table, "cu": cu.int(), "lens": torch.where(ok, ctx + new, 0).int(), "pos": pos.int(),
            "slots": torch.where(live, page * P + pos % P, -1),
            "next": (head + torch.where(ok, upto, 0).amax()).int().reshape(1)}


def _exponent(amax):
    """Least E with amax <= 448 * 2^E, held in [E_MIN, E_MAX]."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _plain_store(s):
    c = s["case"]
    P, H, D = c["P"], c["Hkv"], c["D"]
    codes, scales = _views(s["pool"], c)
    pages = codes.shape[0]
    slots = s["slots"]
    blocks = pages * P // BLOCK
    live = (slots >= 0) & (slots < pages * P)
    blk = torch.where(live, slots // BLOCK, blocks)  # rows that are not stored go to a block of their own
    kv = torch.stack([s["k"].float(), s["v"].float()], dim=2)  # [n, Hkv, 2, D]
    mag = torch.where(torch.isfinite(kv), kv.abs(), 0.0).amax(-1)
    amax = mag.new_zeros(blocks + 1, H, 2)
    amax.scatter_reduce_(0, blk[:, None, None].expand(-1, H, 2), mag, "amax")
    first = torch.full((blocks + 1,), BLOCK, device=slots.device)
    first.scatter_reduce_(0, blk, slots.clamp(min=0) % BLOCK, "amin")
    first = first[:blocks].view(pages, 1, P // BLOCK, 1)
    new_e = _exponent(amax[:blocks]).view(pages, P // BLOCK, H, 2).transpose(1, 2)
    old_e = scales.int() - 127
    e = torch.where(first < BLOCK, torch.where(first > 0, torch.maximum(old_e, new_e), new_e), old_e)
    # what the block held before the call's first slot takes the block's new scale
    off = (torch.arange(P, device=slots.device) % BLOCK).view(1, 1, P // BLOCK, BLOCK, 1, 1)
    held = codes.reshape(pages, H, P // BLOCK, BLOCK, 2, D)
    moved = (first[..., None, None] < BLOCK) & (off < first[..., None, None])
    gain = _pow2((old_e - e).clamp(-126, 0))[:, :, :, None, :, None]
    moved = torch.where(moved, _codes(held.view(torch.float8_e4m3fn).float() * gain).view(torch.uint8), held)
    whole = torch.cat([moved.view(pages, H, P, 2, D), moved.new_zeros(1, H, P, 2, D)])
    page = torch.where(live, slots // P, pages)
    at = slots.clamp(min=0) % P
    row_e = e[page.clamp(max=pages - 1), :, at // BLOCK]  # [n, Hkv, 2]
    x = torch.where(torch.isnan(kv), 0.0, kv) * _pow2(-row_e)[..., None]
    whole[page, :, at] = _codes(x).view(torch.uint8)
    return {"codes": whole[:pages].view(torch.float8_e4m3fn), "scales": (e + 127).to(torch.uint8)}


def _softmax_sum(q, k, v, see, scale):
    """q [.., M, D], k and v [.., N, D], see [.., M or 1, N]: outputs and ln of the sums."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, 1.0)
    return o, (top + total.log())[..., 0]


def _plain_attention(s):
    c = s["case"]
    P, H, D, T, B = c["P"], c["Hkv"], c["D"], s["T"], c["B"]
    G = c["Hq"] // H
    codes, scales = _views(s["pool"], c)
    dev = codes.device
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    i = t - cu[b]
    nq = cu[1:] - cu[:-1]
    vis = (lens[b] - nq[b] + i + 1).clamp(min=0) if c["causal"] else lens[b]
    vis = torch.where(live, torch.minimum(vis, lens[b]), 0)
    if s["sel"] is not None:
        at = s["sel"].long()
        see = (at >= 0) & (at < vis[:, None])
        at = torch.where(see, at, 0)
        page = s["table"][b[:, None], at // P].long().clamp(min=0)
        kv, e = codes[page, :, at % P], scales[page, :, at % P // BLOCK]
    else:
        at = torch.arange(s["max_k"], device=dev)
        page = s["table"][:, at // P].long().clamp(min=0)
        kv, e = codes[page, :, at % P], scales[page, :, at % P // BLOCK]
        see = at < lens[:, None]
    # kv [n, keys, Hkv, 2, D]; keys that nobody sees are taken as zeros
    kv = kv.view(torch.float8_e4m3fn).float().mul_(_pow2(e.int() - 127)[..., None])
    kv = kv.masked_fill_(~see[:, :, None, None, None], 0.0)
    k, v = kv[..., 0, :].transpose(1, 2), kv[..., 1, :].transpose(1, 2)  # [n, Hkv, keys, D]
    q = s["q"].float().view(T, H, G, D)
    if s["sel"] is not None:
        o, lse = _softmax_sum(q, k, v, see[:, None, None, :], s["scale"])  # [T, Hkv, G, D]
    else:
        j = torch.arange(s["max_q"], device=dev)
        rows = (cu[:-1, None] + j).clamp(max=T - 1)
        q = q[rows].permute(0, 2, 3, 1, 4).reshape(B, H, G * s["max_q"], D)
        see = (at < vis[rows][..., None]).repeat(1, G, 1)[:, None]
        o, lse = _softmax_sum(q, k, v, see, s["scale"])
        o = o.view(B, H, G, s["max_q"], D)[b, :, :, i.clamp(max=s["max_q"] - 1)]
        lse = lse.view(B, H, G, s["max_q"])[b, :, :, i.clamp(max=s["max_q"] - 1)]
    o = o.reshape(T, c["Hq"], D).to(s["out"].dtype)
    lse = lse.reshape(T, c["Hq"])
    # rows behind the last sequence stay as they were
    return {"out": torch.where(live[:, None, None], o, s["out"]), "lse": torch.where(live[:, None], lse, s["lse"])}


# ------------------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    if c["op"] == "step_meta":
        return None  # whole numbers only
    s = prepare(c, seed)
    return _exact_store(s) if c["op"] == "kv_store" else _exact_attention(s)


def _e4m3_table():
    """The 256 values of e4m3, from its definition."""
    vals = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        vals.append(-x if byte >> 7 else x)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, saturating, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    step = torch.where(x.abs() < 8 * step, step / 2, step)  # a log2 that came out one too high
    step = torch.where(x.abs() >= 16 * step, step * 2, step).clamp(min=2.0 ** -9)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_store(s):
    c = s["case"]
    P, H = c["P"], c["Hkv"]
    codes, scales = _views(s["pool"], c)
    val = _e4m3_table()[codes.long()]
    exps = scales.double() - 127
    slots = s["slots"].tolist()
    order = [r for r in range(len(slots)) if 0 <= slots[r] < val.shape[0] * P]
    groups, last = [], None
    for r in order:
        if slots[r] // BLOCK != last:
            groups.append([])
            last = slots[r] // BLOCK
        groups[-1].append(r)
    if len(groups) > 4000:
        return None
    kv = torch.stack([s["k"], s["v"]], dim=2).double()
    for g in groups:
        page, at = slots[g[0]] // P, slots[g[0]] % P
        i, f = at // BLOCK, at % BLOCK
        x = kv[g[0]:g[-1] + 1].transpose(0, 1)  # [Hkv, rows, 2, D]
        amax = x.abs().amax((1, 3))
        e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -60) / 448.0))
        e = torch.where(448.0 * torch.exp2(e - 1) >= amax, e - 1, e)
        e = torch.where(448.0 * torch.exp2(e) < amax, e + 1, e).clamp(E_MIN, E_MAX)
        if f:
            old = exps[page, :, i].clone()
            e = torch.maximum(old, e)
            lo = slice(i * BLOCK, i * BLOCK + f)
            val[page, :, lo] = _round_e4m3(val[page, :, lo] * torch.exp2(old - e)[:, None, :, None])
        exps[page, :, i] = e
        val[page, :, at:at + len(g)] = _round_e4m3(x * torch.exp2(-e)[:, None, :, None])
    return {"codes": val, "scales": (exps + 127).to(torch.uint8)}


def _exact_attention(s):
    c = s["case"]
    P, H, D = c["P"], c["Hkv"], c["D"]
    G = c["Hq"] // H
    codes, scales = _views(s["pool"], c)
    table = _e4m3_table()
    out = s["out"].double()
    lse = s["lse"].double()
    cu, t0 = s["cu"].tolist(), 0
    for b, (n, rows) in enumerate(zip(s["lens"].tolist(), _visible(c))):
        t0 = cu[b]
        if not rows:
            continue
        pos = torch.arange(n, device="cuda")
        page = s["table"][b, pos // P].long()
        vis = torch.tensor(rows, device="cuda")
        for h in range(H):
            kv = table[codes[page, h, pos % P].long()]
            kv = kv * torch.exp2(scales[page, h, pos % P // BLOCK].double() - 127)[..., None]
            step = max(1, (1 << 27) // max(1, G * n)) if not c["k"] else max(1, (1 << 27) // (c["k"] * D * 2))
            for a in range(0, len(rows), step):
                z = min(len(rows), a + step)
                q = s["q"][t0 + a:t0 + z, h * G:(h + 1) * G].double()  # [r, G, D]
                if c["k"]:
                    at = s["sel"][t0 + a:t0 + z].long()
                    see = ((at >= 0) & (at < vis[a:z, None]))[:, None]
                    pick = kv[at.clamp(0, n - 1)] if n else kv.new_zeros(z - a, at.shape[1], 2, D)
                    x = torch.einsum("rgd,rkd->rgk", q, pick[:, :, 0]) * s["scale"]
                else:
                    see = (pos < vis[a:z, None])[:, None]
                    x = torch.einsum("rgd,kd->rgk", q, kv[:, 0]) * s["scale"]
                x = torch.where(see, x, -math.inf)
                l = torch.logsumexp(x, -1) if x.shape[-1] else x.new_full(x.shape[:2], -math.inf)
                p = torch.where(see, torch.exp(x - torch.where(l > -math.inf, l, 0.0)[..., None]), 0.0)
                o = torch.einsum("rgk,rkd->rgd", p, pick[:, :, 1]) if c["k"] else torch.einsum("rgk,kd->rgd", p, kv[:, 1])
                out[t0 + a:t0 + z, h * G:(h + 1) * G] = o
                lse[t0 + a:t0 + z, h * G:(h + 1) * G] = l
    return {"out": out, "lse": lse}
