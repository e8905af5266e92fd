"""Performance cases of what a serving step with drafted tokens needs around the paged caches.

Five operators, used together:

* ``tree``    -- attention of a tree of drafted tokens over the 8-bit paged cache: every cached key in
  front of the tree and the nodes that a row's mask shows, or a list of cached keys and those nodes;
* ``verify``  -- the walk through the tree that accepts drafted tokens by the target's probabilities and
  given random numbers, and the draw of the token behind the last accepted one;
* ``compact`` -- the accepted tokens' rows moved together in the 8-bit cache or in the indexer's cache;
* ``pages``   -- next rows of a page table out of the present ones: forks, cuts, ends, with the pages'
  holders, the list of free pages and the pages that have to be copied;
* ``copy``    -- copies of whole pages.

``run`` computes an operator with elementary torch operations while ``own`` is false, and by the
library's entry points while it is true. Lengths and the trees' shapes are functions of the case alone;
values come from the seed. Node 0 of a sequence's rows is its last accepted token, whose key is the first
that the step adds.

8-bit cache page, as both sides read it: kv head h of a page starts at h * (2*P*D + 16) bytes; token s of
the head has its D K codes at s*2*D and its D V codes right behind them; the scale bytes (exponent + 127)
of 16-token block i are at 2*P*D + 2*i (K) and 2*P*D + 2*i + 1 (V). Indexer's cache page: FP8 token s has
8 chunks of 16 bytes at (s/8)*1024 + c*128 + (s%8)*16 and its fp32 scale at 128*P + 4*s; MXFP4 4 chunks and 4
scale bytes, at the places that ``_token_bytes`` gives.
"""
import math

import torch

own = False

BLOCK = 16                 # tokens of a scale block
WORKSPACE = 64 << 20       # bytes a program keeps for the attention's partial results
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8, MXFP4 = 1, 0          # the library's numbers of the indexer's cache types


# ------------------------------------------------------------------------------ cases

def listed():
    tree = dict(op="tree", type="bf16", D=128, P=128, k=0, pad=0, empty_every=0, hole_every=0)
    return [
        # one short request with a small tree: latency alone
        dict(tree, name="tree_one", type="fp16", B=1, Hq=8, Hkv=1, q_lo=8, q_hi=8, fan=3, ctx_lo=504, ctx_hi=504),
        # a drafting step of 64 requests with full caches, 16 nodes each
        dict(tree, name="tree_decode_64", B=64, Hq=64, Hkv=8, q_lo=16, q_hi=16, fan=4, ctx_lo=8176, ctx_hi=8176),
        # trees of unlike sizes, padded nodes that see nothing of the tree, padded rows, odd heads
        dict(tree, name="tree_ragged_odd", type="fp16", B=9, Hq=12, Hkv=4, D=64, P=64, q_lo=1, q_hi=67, fan=5, ctx_lo=0,
             ctx_hi=3001, pad=7, hole_every=6),
        # a sparse layer's drafting step: the indexer's 1024 cached keys per node, 64 heads that share the cache
        dict(tree, name="tree_topk_64", B=64, Hq=64, Hkv=1, q_lo=8, q_hi=8, fan=3, ctx_lo=8184, ctx_hi=8184, k=1024),
        # one request, a chain of four drafted tokens without the drafter's probabilities, an odd vocabulary
        dict(op="verify", name="verify_one", type="bf16", B=1, V=49999, q_lo=5, q_hi=5, fan=1, drafter=0, most=8),
        # 64 trees of 32 nodes by both sides' probabilities, a large vocabulary
        dict(op="verify", name="verify_tree_64", type="fp32", B=64, V=131072, q_lo=32, q_hi=32, fan=4, drafter=1, most=12),
        # accepted tokens of 64 requests, 8 layers of the 8-bit cache
        dict(op="compact", name="compact_kv_64", cache="kv", B=64, Hkv=8, D=128, P=128, layers=8, q_lo=16, q_hi=16,
             ctx_lo=0, ctx_hi=500, most=6),
        # the same in the indexer's cache of one layer
        dict(op="compact", name="compact_indexer_64", cache="fp8", B=64, Hkv=1, D=128, P=64, layers=1, q_lo=1, q_hi=33,
             ctx_lo=0, ctx_hi=900, most=9),
        # a step's end of 64 requests: rejected tokens' pages go back
        dict(op="pages", name="pages_step_64", B=64, out=64, P=128, ctx_lo=1, ctx_hi=8192, kind="cut", group=1, spare=2000,
             short=0),
        # many requests, prompts shared in groups, beams that fork and end
        dict(op="pages", name="pages_beams_1024", B=1024, out=1024, P=64, ctx_lo=0, ctx_hi=16000, kind="mixed", group=4,
             spare=70000, short=0),
        # four pages of one layer
        dict(op="copy", name="copy_4", n=4, skip_every=0, page=8 * 32784, layers=1),
        # the last pages of 64 forked requests, every third row without a copy, 16 layers
        dict(op="copy", name="copy_64_layers", n=64, skip_every=3, page=8 * 32784, layers=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "compact", "pages", "copy"])
    if op == "tree":
        k = rng.choice([0, 0, 32, 257, 1024, 2048])
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 1, 2, 4] if k else [1, 2, 3, 4, 8])
        group = rng.choice([4, 8, 16, 32, 64] if k and Hkv == 1 else [1, 2, 4, 7, 8, 16])
        q_hi = _log(rng, 1, max(2, min(100, (400 if k else 1000) // B)))
        ctx = _log(rng, 1, max(2, min(60000, 20000 if k else 500000000 // (B * q_hi * Hkv * group))))
        return dict(op=op, type=rng.choice(["bf16", "fp16"]), D=rng.choice([64, 128]), P=rng.choice([64, 128]), B=B, Hkv=Hkv,
                    Hq=Hkv * group, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, fan=rng.choice([1, 2, 4, 9]),
                    ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx, k=k, pad=rng.choice([0, 0, 5]),
                    empty_every=rng.choice([0, 0, 3]), hole_every=rng.choice([0, 0, 4]))
    if op == "verify":
        V = _log(rng, 1000, 131072)
        B = _log(rng, 1, 64)
        q_hi = _log(rng, 1, 32)
        return dict(op=op, type=rng.choice(["fp32", "fp32", "bf16", "fp16"]), B=B, V=V, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi,
                    fan=rng.choice([1, 2, 4]), drafter=rng.choice([0, 1, 1]), most=rng.choice([3, 9, 33]))
    if op == "compact":
        q_hi = _log(rng, 1, 70)
        return dict(op=op, cache=rng.choice(["kv", "kv", "fp8", "mxfp4"]), B=_log(rng, 1, 100), Hkv=rng.choice([1, 2, 3, 8]),
                    D=rng.choice([64, 128]), P=rng.choice([64, 128]), layers=rng.choice([1, 1, 2, 5]), q_lo=rng.choice([0, 1, q_hi]),
                    q_hi=q_hi, ctx_lo=0, ctx_hi=_log(rng, 1, 700), most=rng.choice([1, 5, 40]))
    if op == "pages":
        B = _log(rng, 1, 1024)
        kind = rng.choice(["cut", "fork", "mixed"])
        return dict(op=op, B=B, out=max(1, B if kind == "cut" else rng.choice([B, B // 2, min(1024, 3 * B)])), P=rng.choice([64, 128]), ctx_lo=0,
                    ctx_hi=_log(rng, 1, max(2, min(16000, 12000000 // B))), kind=kind, group=rng.choice([1, 1, 3, 8]),
                    spare=_log(rng, 1, 50000), short=rng.choice([0, 0, 1]))
    return dict(op=op, n=_log(rng, 1, 64), skip_every=rng.choice([0, 2, 5]), page=16 * _log(rng, 256, 16000), layers=rng.choice([1, 3, 12]))


def _hash(i, salt):
    return (i + salt) * 2654435761 % 4294967296 >> 7


def _ragged(n, lo, hi, salt):
    """n lengths in [lo, hi], spread but fixed: a function of the arguments alone."""
    return [lo + _hash(i, salt) % (hi - lo + 1) for i in range(n)]


def _lengths(c):
    ctx = _ragged(c["B"], c.get("ctx_lo", 0), c.get("ctx_hi", 0), 11)
    new = _ragged(c["B"], c["q_lo"], c["q_hi"], 5)
    if sum(new) == 0:
        new[0] = 1
    return ctx, new


def _seq_lens(c):
    """Keys of each sequence of a tree case; some have none although they have rows."""
    ctx, new = _lengths(c)
    e = c["empty_every"]
    return [0 if e and b % e == e - 1 else x + y for b, (x, y) in enumerate(zip(ctx, new))]


def _parents(n, fan, salt):
    """A tree of n nodes, parents in front of their children; fan 1: a chain."""
    return [-1 if j == 0 else j - 1 - _hash(j, salt) % min(j, fan) for j in range(n)]


def _masks(c):
    """For each row the nodes that it sees, as a whole number, sequence after sequence."""
    _, new = _lengths(c)
    rows = []
    for b, n in enumerate(new):
        seen = []
        for j, p in enumerate(_parents(n, c["fan"], b)):
            seen.append(1 << j | (seen[p] if p >= 0 else 0))
        h = c["hole_every"]
        rows += [0 if h and j % h == h - 1 else m for j, m in enumerate(seen)]
    return rows


def _path_lens(c):
    """Accepted nodes of each request of a compact case."""
    _, new = _lengths(c)
    return [min(n, 1 + _hash(b, 3) % c["most"]) for b, n in enumerate(new)]


def _page_rows(c):
    """A pages case: lengths of the present rows, parent and tokens kept of the next ones."""
    lens = _ragged(c["B"], c["ctx_lo"], c["ctx_hi"], 11)
    parent, keep = [], []
    for b in range(c["out"]):
        if c["kind"] == "cut":
            p = b
            k = max(0, lens[p] - _hash(b, 2) % 16)
        elif c["kind"] == "fork":
            p = b * c["B"] // c["out"]
            k = lens[p]
        else:
            p = _hash(b, 21) % (c["B"] + 1) - 1
            k = 0 if p < 0 else lens[p] if _hash(b, 4) % 3 else _hash(b, 8) % (lens[p] + 1)
        parent.append(p)
        keep.append(k)
    return lens, parent, keep


def work(c):
    if c["op"] == "copy":
        n = sum(1 for i in range(c["n"]) if not _skipped(c, i))
        return {"bytes": 2 * n * c["page"] * c["layers"] + 8 * c["n"], "flops": 0}
    if c["op"] == "pages":
        lens, parent, keep = _page_rows(c)
        held, kept = sum(-(-n // c["P"]) for n in lens), sum(-(-n // c["P"]) for n in keep)
        return {"bytes": 4 * (held + kept + 2 * (held + c["spare"]) + 2 * c["spare"] + c["B"] + 5 * c["out"]), "flops": 0}
    ctx, new = _lengths(c)
    if c["op"] == "compact":
        token = c["Hkv"] * (2 * c["D"] + 0.125) if c["cache"] == "kv" else 132 if c["cache"] == "fp8" else 68
        return {"bytes": 2 * c["layers"] * token * sum(max(0, n - 1) for n in _path_lens(c)) + 4 * sum(_path_lens(c)) + 12 * c["B"],
                "flops": 0}
    if c["op"] == "verify":  # the row that the last token is drawn from, of either side
        size = 4 if c["type"] == "fp32" else 2
        live = sum(1 for n in new if n)
        return {"bytes": live * c["V"] * size * (1 + c["drafter"]) + 12 * sum(new) + 8 * c["B"] * c["most"],
                "flops": live * c["V"] * (1 + 2 * c["drafter"])}
    seen, keys, row = 0, 0, 0
    masks = _masks(c)
    for n, q in zip(_seq_lens(c), new):
        front = max(n - q, 0)
        per = min(front, c["k"]) if c["k"] else front
        seen += sum(per + (bin(m).count("1") if n >= q else 0) for m in masks[row:row + q])
        keys += (min(front, per * q) if c["k"] else front) + min(q, n) if q else 0
        row += q
    rows = sum(new)
    return {"bytes": keys * c["Hkv"] * (2 * c["D"] + 0.125) + rows * (c["Hq"] * (4 * c["D"] + 4) + 4 * c["k"] + -(-c["q_hi"] // 64) * 8),
            "flops": 4 * c["D"] * c["Hq"] * seen}


def _skipped(c, i):
    return bool(c["skip_every"]) and i % c["skip_every"] == c["skip_every"] - 1


# ------------------------------------------------------------------------------ inputs

def _views(pool, c):
    """Codes [.., pages, Hkv, P, 2, D] and scale bytes [.., pages, Hkv, P/16, 2] of a pool, in place."""
    H, P, D = c["Hkv"], c["P"], c["D"]
    head = 2 * P * D + 16
    lead, st = tuple(pool.shape[:-1]), pool.stride()[:-1]
    codes = pool.as_strided((*lead, H, P, 2, D), (*st, head, 2 * D, D, 1))
    scales = pool.as_strided((*lead, H, P // BLOCK, 2), (*st, head, 2, 1), 2 * P * D)
    return codes, scales


def _pages(lens, P, spare, gen, width):
    """A shuffled page table [B, width] (-1 where there is no page) and how many pages there are."""
    need = [-(-n // P) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    start = need_t.cumsum(0) - need_t
    j = torch.arange(width, device="cuda")
    at = (start[:, None] + j).clamp(max=total - 1)
    return torch.where(j < need_t[:, None], perm[at], -1).to(torch.int32).contiguous(), total


def _fill(pool, c, gen):
    """Codes and scales as the store leaves them."""
    codes, scales = _views(pool, c)
    x = torch.empty(codes.shape, device="cuda", dtype=torch.bfloat16).normal_(0.0, 100.0, generator=gen)
    codes.copy_(x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    scales.copy_(torch.randint(119, 123, scales.shape, generator=gen, device="cuda", dtype=torch.uint8))


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    return {"tree": _prepare_tree, "verify": _prepare_verify, "compact": _prepare_compact, "pages": _prepare_pages,
            "copy": _prepare_copy}[c["op"]](c, gen)


I32 = dict(dtype=torch.int32, device="cuda")


def _cu(new):
    return torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)


def _prepare_tree(c, gen):
    ctx, new = _lengths(c)
    lens, T, P = _seq_lens(c), sum(new) + c["pad"], c["P"]
    width = max(1, -(-max(lens) // P))
    table, pages = _pages(lens, P, 2, gen, width)
    pool = torch.zeros(pages, c["Hkv"] * (2 * P * c["D"] + 16), dtype=torch.uint8, device="cuda")
    _fill(pool, c, gen)
    dt, lens_t = TYPES[c["type"]], torch.tensor(lens, **I32)
    # slots past a sequence's length hold what earlier requests left, NaN codes here
    codes, _ = _views(pool, c)
    last = ((lens_t.long() - 1).clamp(min=0) // P).clamp(max=width - 1)
    page = table.gather(1, last[:, None])[:, 0].long().clamp(min=0)
    stale = (torch.arange(P, device="cuda") >= (lens_t.long() - last * P)[:, None]) & (lens_t > 0)[:, None]
    codes[page] = torch.where(stale[:, None, :, None, None], 127, codes[page])
    words = -(-max(new) // 64)
    masks = [[m >> 64 * w & (1 << 64) - 1 for w in range(words)] for m in _masks(c)] + [[0] * words] * c["pad"]
    masks = [[x - (1 << 64) if x >> 63 else x for x in row] for row in masks]
    s = {"case": c, "T": T, "pool": pool, "table": table, "lens": lens_t, "cu": _cu(new), "max_q": max(new), "max_k": max(1, *lens),
         "mask": torch.tensor(masks, dtype=torch.int64, device="cuda").reshape(T, words),
         "q": torch.randn(T, c["Hq"], c["D"], generator=gen, device="cuda").to(dt), "scale": c["D"] ** -0.5,
         "out": torch.zeros(T, c["Hq"], c["D"], dtype=dt, device="cuda"), "lse": torch.zeros(T, c["Hq"], device="cuda"),
         "workspace": torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda"), "sel": None,
         "status": torch.zeros(1, **I32)}
    if c["k"]:  # k distinct keys in front of the tree per row, by random keys
        front = torch.tensor([max(n - q, 0) for n, q in zip(lens, new) for _ in range(q)] + [0] * c["pad"], device="cuda")
        most = max(1, max(x for x in ctx))
        n = min(c["k"], most)
        sel = torch.full((T, c["k"]), -1, **I32)
        rows = max(1, (1 << 28) // most)
        for at in range(0, T, rows):
            v = front[at:at + rows, None]
            r = torch.rand(v.shape[0], most, generator=gen, device="cuda")
            top, idx = torch.where(torch.arange(most, device="cuda") < v, r, -1.0).topk(n, dim=1)
            sel[at:at + rows, :n] = torch.where(top >= 0, idx, -1).to(torch.int32)
        s["sel"] = sel
    return s


def _prepare_verify(c, gen):
    _, new = _lengths(c)
    T, V, dt = sum(new), c["V"], TYPES[c["type"]]
    target, draft = torch.empty(T, V, dtype=dt, device="cuda"), torch.empty(T, V, dtype=dt, device="cuda")
    rows = max(1, (1 << 27) // V)
    for at in range(0, T, rows):  # the drafter's logits follow the target's
        z = torch.randn(min(rows, T - at), V, generator=gen, device="cuda") * 3.0
        target[at:at + rows] = z.softmax(-1)
        z = z * 0.9 + torch.randn(z.shape, generator=gen, device="cuda") * 0.7
        draft[at:at + rows] = z.softmax(-1)
    parents = [p for b, n in enumerate(new) for p in _parents(n, c["fan"], b)]
    first = [sum(new[:b]) for b, n in enumerate(new) for _ in range(n)]
    up = torch.tensor([f + max(p, 0) for f, p in zip(first, parents)], device="cuda")
    tokens = torch.empty(T, **I32)
    for at in range(0, T, rows):  # each node drawn from the drafter's probabilities behind its parent
        w = draft[up[at:at + rows]].float()
        tokens[at:at + rows] = (w / torch.empty_like(w).exponential_(generator=gen).clamp_(min=1e-30)).argmax(-1).to(torch.int32)
    return {"case": c, "target": target, "draft": draft if c["drafter"] else None, "tokens": tokens,
            "parents": torch.tensor(parents, **I32), "coins": torch.rand(T, generator=gen, device="cuda"),
            "last": torch.rand(c["B"], generator=gen, device="cuda"), "cu": _cu(new), "max_q": max(new),
            "path": torch.full((c["B"], c["most"]), -7, **I32), "n_path": torch.full((c["B"],), -7, **I32),
            "out": torch.full((c["B"], c["most"]), -7, **I32), "status": torch.zeros(1, **I32)}


def _page_bytes(c):
    return c["Hkv"] * (2 * c["P"] * c["D"] + 16) if c["cache"] == "kv" else c["P"] * (132 if c["cache"] == "fp8" else 68)


def _prepare_compact(c, gen):
    ctx, new = _lengths(c)
    lens = [x + y for x, y in zip(ctx, new)]
    table, pages = _pages(lens, c["P"], 2, gen, max(1, -(-max(lens) // c["P"])))
    pool = torch.randint(0, 127, (c["layers"], pages + 1, _page_bytes(c)), generator=gen, device="cuda", dtype=torch.uint8)
    if c["cache"] == "kv":
        _fill(pool, c, gen)
    n_path = torch.tensor(_path_lens(c), device="cuda")
    # the accepted nodes: node 0 and n_path - 1 others, in order
    r = torch.rand(c["B"], max(new), generator=gen, device="cuda")
    node = torch.arange(max(new), device="cuda")
    r = torch.where(node < torch.tensor(new, device="cuda")[:, None], r, 2.0)
    r[:, 0] = -1.0
    rank = r.argsort(1).argsort(1)
    order = torch.where(rank < n_path[:, None], node, 1 << 20).sort(1).values
    most = max(_path_lens(c) + [1])
    path = torch.where(order < 1 << 20, order, -1)[:, :most].to(torch.int32).contiguous()
    return {"case": c, "pool": pool, "table": table, "lens": torch.tensor(lens, **I32), "cu": _cu(new), "path": path,
            "n_path": n_path.to(torch.int32), "new_lens": torch.zeros(c["B"], **I32), "status": torch.zeros(1, **I32)}


def _prepare_pages(c, gen):
    lens, parent, keep = _page_rows(c)
    B, P, g = c["B"], c["P"], c["group"]
    width = max(1, -(-max(lens) // P))
    lens_t = torch.tensor(lens, device="cuda")
    held = (lens_t + P - 1) // P
    j = torch.arange(width, device="cuda")
    # the rows of a group hold the same pages up to half of its shortest row
    b = torch.arange(B, device="cuda")
    lead = b - b % g
    shortest = torch.full((B,), 1 << 30, device="cuda").scatter_reduce_(0, lead, lens_t, "amin")[lead]
    mine = (j < held[:, None]) & ((b == lead)[:, None] | (j >= (shortest // 2 // P)[:, None]))
    ids = mine.view(-1).cumsum(0).view(B, width) - 1
    pages = int(mine.sum()) + c["spare"]
    perm = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    own_id = torch.where(mine, perm[ids.clamp(min=0)], -1)
    table = torch.where(mine, own_id, torch.where(j < held[:, None], own_id[lead], -1)).to(torch.int32).contiguous()
    held_by = torch.bincount(table[table >= 0].long(), minlength=pages)
    free = torch.full((pages,), -1, **I32)
    head = 3 if c["spare"] > 5 else 0
    free[head:c["spare"]] = perm[pages - c["spare"] + head:]
    span = [head, min(c["spare"], head + 1 + c["out"] // 8) if c["short"] else c["spare"]]
    return {"case": c, "parent": torch.tensor(parent, **I32), "keep": torch.tensor(keep, **I32), "table": table,
            "lens": torch.tensor(lens, **I32), "shares": (held_by - 1).clamp(min=0).to(torch.int32), "free": free,
            "span": torch.tensor(span, **I32), "new_table": torch.full((c["out"], width), -1, **I32),
            "new_lens": torch.zeros(c["out"], **I32), "new_shares": torch.zeros(pages, **I32), "new_free": torch.full((pages,), -1, **I32),
            "new_span": torch.zeros(2, **I32), "copies": torch.zeros(c["out"], 2, **I32), "status": torch.zeros(1, **I32)}


def _prepare_copy(c, gen):
    n = c["n"]
    perm = torch.randperm(2 * n + 3, generator=gen, device="cuda").to(torch.int32)
    pairs = torch.stack([perm[:n], perm[n:2 * n]], 1)
    skip = torch.tensor([_skipped(c, i) for i in range(n)], device="cuda")
    pool = torch.randint(0, 256, (c["layers"], 2 * n + 3, c["page"]), generator=gen, device="cuda", dtype=torch.uint8)
    return {"case": c, "pool": pool, "pairs": torch.where(skip[:, None], -1, pairs).contiguous(), "status": torch.zeros(1, **I32)}


# ------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"tree": _own_tree, "verify": _own_verify, "compact": _own_compact, "pages": _own_pages, "copy": _own_copy}[op](s)
    return {"tree": _plain_tree, "verify": _plain_verify, "compact": _plain_compact, "pages": _plain_pages,
            "copy": _plain_copy}[op](s)


def _own_tree(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    c = s["case"]
    idx.idx_attn_tree(s["q"], s["pool"], s["pool"].shape[0], c["P"], s["pool"].stride(0), c["Hkv"], s["table"], s["lens"],
                      s["cu"], s["mask"], s["max_q"], s["max_k"], s["scale"], s["out"], lse=s["lse"], sel_idx=s["sel"],
                      workspace=s["workspace"], dev_status=s["status"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_verify(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    idx.idx_draft_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["coins"], s["last"], s["cu"], s["max_q"],
                         s["path"], s["n_path"], s["out"], dev_status=s["status"])
    return {"path": s["path"], "n_path": s["n_path"], "tokens": s["out"]}


def _own_compact(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    c, pool = s["case"], s["pool"]
    if c["cache"] == "kv":
        idx.idx_kv_compact(s["path"], s["n_path"], s["lens"], s["cu"], s["table"], pool, pool.shape[1], c["P"], pool.stride(1),
                           c["Hkv"], c["D"], layers=c["layers"], layer_stride=pool.stride(0), new_lens=s["new_lens"],
                           dev_status=s["status"])
    else:
        idx.idx_k_compact(s["path"], s["n_path"], s["lens"], s["cu"], s["table"], FP8 if c["cache"] == "fp8" else MXFP4, pool,
                          pool.shape[1], c["P"], pool.stride(1), layers=c["layers"], layer_stride=pool.stride(0),
                          new_lens=s["new_lens"], dev_status=s["status"])
    return _compact_outputs(s, s["new_lens"])


def _own_pages(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    idx.idx_pages_update(s["parent"], s["keep"], s["table"], s["lens"], s["case"]["P"], s["new_table"], s["new_lens"], s["shares"],
                         s["new_shares"], s["free"], s["span"], s["new_free"], s["new_span"], s["copies"], dev_status=s["status"])
    return {k: s[k] for k in ("new_table", "new_lens", "new_shares", "new_free", "new_span", "copies")}


def _own_copy(s):
    from sparse_attention_indexer_mqa_gb300 import binding as idx
    c, pool = s["case"], s["pool"]
    idx.idx_pages_copy(s["pairs"], pool, pool.shape[1], c["page"], pool.stride(1), layers=c["layers"], layer_stride=pool.stride(0),
                       dev_status=s["status"])
    return pool


# ------------------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e in 32 bits for whole e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _softmax_sum(q, k, v, see, scale):
    """q [.., M, D], k and v [.., N, D], see [.., M or 1, N]: outputs and ln of the sums."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total > 0, total, 1.0)
    return o, (top + total.log())[..., 0]


def _plain_tree(s):
    c = s["case"]
    P, H, D, T, B, N = c["P"], c["Hkv"], c["D"], s["T"], c["B"], s["max_q"]
    G = c["Hq"] // H
    codes, scales = _views(s["pool"], c)
    dev = codes.device
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    i, nq = t - cu[b], cu[1:] - cu[:-1]
    front = lens - nq  # position of a sequence's node 0
    node = torch.arange(N, device=dev)
    bits = (s["mask"][:, node // 64] >> node % 64 & 1).bool() & (node < nq[b][:, None]) & live[:, None]  # [T, N]
    q = s["q"].float().view(T, H, G, D)
    if s["sel"] is not None:
        at = s["sel"].long()
        see = torch.cat([(at >= 0) & (at < front[b][:, None]) & live[:, None], bits & (front[b][:, None] + node >= 0)], 1)
        at = torch.where(see, torch.cat([at, front[b][:, None] + node], 1), 0)
        page = s["table"][b[:, None], at // P].long().clamp(min=0)
    else:
        at = torch.arange(s["max_k"], device=dev)
        page = s["table"][:, at // P].long().clamp(min=0)
        see = at < lens[:, None]
    # kv [n, keys, Hkv, 2, D]; keys that nobody sees are taken as zeros
    kv = codes[page, :, at % P].view(torch.float8_e4m3fn).float()
    kv = kv.mul_(_pow2(scales[page, :, at % P // BLOCK].int() - 127)[..., None]).masked_fill_(~see[:, :, None, None, None], 0.0)
    k, v = kv[..., 0, :].transpose(1, 2), kv[..., 1, :].transpose(1, 2)  # [n, Hkv, keys, D]
    if s["sel"] is not None:
        o, lse = _softmax_sum(q, k, v, see[:, None, None, :], s["scale"])  # [T, Hkv, G, D]
    else:
        rows = (cu[:-1, None] + node).clamp(max=T - 1)  # [B, N]
        q = q[rows].permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
        at_node = at - front[:, None]  # [B, keys]
        shown = bits[rows].gather(2, at_node.clamp(0, N - 1)[:, None].expand(-1, N, -1))
        shown = torch.where(at_node[:, None] < 0, True, shown) & see[:, None]
        o, lse = _softmax_sum(q, k, v, shown.repeat(1, G, 1)[:, None], s["scale"])
        o = o.view(B, H, G, N, D)[b, :, :, i.clamp(max=N - 1)]
        lse = lse.view(B, H, G, N)[b, :, :, i.clamp(max=N - 1)]
    o = o.reshape(T, c["Hq"], D).to(s["out"].dtype)
    # rows behind the last sequence stay as they were
    return {"out": torch.where(live[:, None, None], o, s["out"]),
            "lse": torch.where(live[:, None], lse.reshape(T, c["Hq"]), s["lse"])}


def _plain_verify(s):
    """Nodes in index order, all requests at once: a node is tested when its parent is where the walk stands. In 64
    bits, for the draw looks for a border among sums of a whole vocabulary."""
    c, p, q = s["case"], s["target"], s["draft"]
    B, V, most = c["B"], c["V"], c["most"]
    cu = s["cu"].long()
    first, n = cu[:-1], cu[1:] - cu[:-1]
    dev, last_row = p.device, p.shape[0] - 1
    slot = torch.arange(most, device=dev)

    def row_of(x, node):
        w = x[(first + node).clamp(max=last_row)].double()
        return torch.where((w > 0) & (w < math.inf), w, 0.0)

    def left(node, cut, gone):
        w = row_of(p, node)
        return torch.where(gone, 0.0, w) if q is None else (w - cut[:, None] * row_of(q, node)).clamp_(min=0.0)

    cur = torch.zeros(B, dtype=torch.int64, device=dev)
    path = torch.where((slot == 0) & (n > 0)[:, None], 0, -1)
    tokens = torch.full((B, most), -1, device=dev)
    length = (n > 0).long()
    cut, mass = torch.zeros(B, dtype=torch.float64, device=dev), torch.ones(B, dtype=torch.float64, device=dev)
    gone = torch.zeros(B, V, dtype=torch.bool, device=dev)
    for j in range(1, s["max_q"]):
        at = (first + j).clamp(max=last_row)
        x = s["tokens"][at].long()
        test = (j < n) & (s["parents"][at] == cur) & (length < most) & (x >= 0) & (x < V)
        x = x.clamp(0, V - 1)
        u, px = s["coins"][at].double(), row_of(p, cur).gather(1, x[:, None])[:, 0]
        if q is None:
            px = torch.where(gone.gather(1, x[:, None])[:, 0], 0.0, px)
            yes = test & (u * mass < px)
            mass = torch.where(test & ~yes, (mass - px).clamp(min=0.0), mass)
            gone = gone.scatter(1, x[:, None], (gone.gather(1, x[:, None])[:, 0] | (test & ~yes))[:, None])
        else:
            qx = row_of(q, cur).gather(1, x[:, None])[:, 0]
            yes = test & (u * qx * mass < px - cut * qx)
            no = test & ~yes
            cut = torch.where(no, cut + mass, cut)
            mass = torch.where(no, left(cur, cut, gone).sum(1), mass)
        here = yes[:, None] & (slot == length[:, None])
        path = torch.where(here, j, path)
        tokens = torch.where(yes[:, None] & (slot == (length - 1)[:, None]), x[:, None], tokens)
        length = length + yes
        cur = torch.where(yes, j, cur)
        cut, mass, gone = torch.where(yes, 0.0, cut), torch.where(yes, 1.0, mass), gone & ~yes[:, None]
    w = left(cur, cut, gone)
    w = torch.where((w.sum(1) > 0)[:, None], w, row_of(p, cur))
    sums = w.cumsum(1)
    drawn = (sums <= s["last"].double()[:, None] * sums[:, -1:]).sum(1)
    drawn = torch.where(sums[:, -1] > 0, drawn, -1)
    tokens = torch.where((slot == (length - 1)[:, None]) & (n > 0)[:, None], drawn[:, None], tokens)
    return {"path": path.int(), "n_path": length.int(), "tokens": tokens.int()}


def _token_bytes(c):
    """[P, n] places in a page of the indexer's cache of each token's bytes."""
    s, P = torch.arange(c["P"], device="cuda")[:, None], c["P"]
    byte = torch.arange(16, device="cuda")
    if c["cache"] == "fp8":
        at = (s // 8 * 1024 + s % 8 * 16)[:, :, None] + torch.arange(8, device="cuda")[:, None] * 128 + byte
        scale = 128 * P + 4 * s + torch.arange(4, device="cuda")
    else:
        chunk = torch.arange(4, device="cuda")
        if P == 128:
            at, scale = (s // 8 * 4 + chunk) * 128 + s % 8 * 16, 8192 + s % 32 * 16 + s // 32 * 4 + chunk
        else:
            at, scale = s // 16 * 1024 + s // 8 % 2 * 512 + chunk * 128 + s % 8 * 16, 4096 + s % 16 * 16 + s // 16 * 4 + chunk
        at = at[:, :, None] + byte
    return torch.cat([at.reshape(P, -1), scale], 1)


def _compact_outputs(s, new_lens):
    c, pool = s["case"], s["pool"]
    if c["cache"] == "kv":
        codes, scales = _views(pool, c)
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "lens": new_lens}
    if c["cache"] == "fp8":
        return {"codes": pool[..., :128 * c["P"]].view(torch.float8_e4m3fn), "scales": pool[..., 128 * c["P"]:].view(torch.int32),
                "lens": new_lens}
    return {"pages": pool, "lens": new_lens}


def _plain_compact(s):
    c, pool, P = s["case"], s["pool"], s["case"]["P"]
    cu, lens = s["cu"].long(), s["lens"].long()
    nq, n = cu[1:] - cu[:-1], s["n_path"].long()
    front = lens - nq
    i = torch.arange(s["path"].shape[1], device=pool.device)
    on = i < n[:, None]
    i = torch.where(on, i, 0)  # rows without an entry repeat their first, and those without any stay as they are
    some = (n > 0)[:, None]
    src = front[:, None] + torch.where(some, s["path"].long().gather(1, i), 0)
    dst = front[:, None] + i
    last = (lens - 1).clamp(min=0)[:, None]
    src, dst = torch.minimum(src, last), torch.minimum(dst, last)
    b = torch.arange(c["B"], device=pool.device)[:, None]
    page = torch.where(s["table"] < 0, pool.shape[1] - 1, s["table"]).long()  # the last page is nobody's
    src_page, dst_page = page[b, src // P], page[b, dst // P]
    new_lens = (front + n).int()
    if c["cache"] != "kv":
        at = _token_bytes(c)
        pool[:, dst_page[..., None], at[dst % P]] = pool[:, src_page[..., None], at[src % P]]
        return _compact_outputs(s, new_lens)
    codes, scales = _views(pool, c)
    e = scales[:, src_page, :, src % P // BLOCK].int()  # [B, i, layers, Hkv, 2]
    raw = codes[:, src_page, :, src % P].view(torch.float8_e4m3fn).float()  # [B, i, layers, Hkv, 2, D]
    # destination blocks, counted from the one that holds the first token; that one may hold kept tokens too
    blk = front % BLOCK
    group = (blk[:, None] + i) // BLOCK
    groups = (s["path"].shape[1] + 2 * BLOCK) // BLOCK
    top = e.new_zeros(c["B"], groups, *e.shape[2:])
    top.scatter_reduce_(1, group[..., None, None, None].expand(e.shape), e, "amax")
    start = torch.minimum(front, last[:, 0])
    page0, blk0 = page[b[:, 0], start // P], start % P // BLOCK
    old = scales[:, page0, :, blk0].int()  # [B, layers, Hkv, 2]
    top[:, 0] = torch.maximum(top[:, 0], torch.where((blk > 0)[:, None, None, None], old, 0))
    top[:, 0] = torch.where((n > 0)[:, None, None, None], top[:, 0], old)
    # kept tokens of the first block
    off = torch.arange(BLOCK, device=pool.device)
    tok = blk0[:, None] * BLOCK + off  # [B, 16]
    held = codes[:, page0[:, None], :, tok]
    gain = _pow2((old - top[:, 0]).clamp(min=-126))[:, None, ..., None]
    moved = (held.view(torch.float8_e4m3fn).float() * gain).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[:, page0[:, None], :, tok] = torch.where((off < blk[:, None])[..., None, None, None, None], moved, held)
    new_e = top.gather(1, group[..., None, None, None].expand(e.shape))
    out = (raw * _pow2((e - new_e).clamp(min=-126))[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[:, dst_page, :, dst % P] = torch.where(some[..., None, None, None, None], out, codes[:, dst_page, :, dst % P])
    scales[:, dst_page, :, dst % P // BLOCK] = torch.where(some[..., None, None, None], new_e, scales[:, dst_page, :, dst % P // BLOCK].int()).to(torch.uint8)
    return _compact_outputs(s, new_lens)


def _plain_pages(s):
    P, table, lens = s["case"]["P"], s["table"].long(), s["lens"].long()
    parent, keep = s["parent"].long(), s["keep"].long()
    B, width = table.shape
    pages = s["shares"].numel()
    j = torch.arange(width, device=table.device)
    ok = (parent >= 0) & (parent < B) & (keep >= 0)
    par = parent.clamp(0, B - 1)
    ok &= keep <= lens[par]
    kept = torch.where(ok, (keep + P - 1) // P, 0)
    rows = table[par]  # [out, width]
    holds = j < kept[:, None]

    def count(ids, on):  # how often each page occurs
        n = torch.zeros(pages + 1, dtype=torch.int64, device=table.device)
        return n.scatter_add_(0, torch.where(on, ids, pages).reshape(-1), torch.ones_like(ids).reshape(-1))[:pages]

    shares = s["shares"].long() - count(table, j < ((lens + P - 1) // P)[:, None]) + count(rows, holds)
    # a last page that is not full is written by its row: with other holders the row gets a page of its own, but for
    # the first of rows that all end in it
    ends = ok & (keep % P > 0)
    last = rows.gather(1, (keep // P).clamp(0, width - 1)[:, None])[:, 0].clamp(0, pages - 1)
    b = torch.arange(parent.numel(), device=table.device)
    lowest = torch.full((pages + 1,), 1 << 30, device=table.device)
    lowest.scatter_reduce_(0, torch.where(ends, last, pages), b, "amin")
    copy = ends & ~((shares[last] + 1 == count(last, ends)[last]) & (lowest[last] == b))
    head, tail = s["span"].long().unbind()
    at = head + copy.cumsum(0) - copy.long()
    none = copy & (at >= tail)  # no page is left for it: an empty row
    copy &= ~none
    fresh = s["free"][at.clamp(0, s["free"].numel() - 1)].long()
    shares = shares - count(last, copy) - count(rows, holds & none[:, None])
    kept = torch.where(none, 0, kept)
    new = torch.where(copy[:, None] & (j == (keep // P)[:, None]), fresh[:, None], rows)
    new_table = torch.where(j < kept[:, None], new, s["new_table"].long())
    freed = shares < 0
    left = (tail - head - copy.sum()).clamp(min=0)
    start = head + copy.sum()
    i = torch.arange(pages, device=table.device)
    new_free = torch.where(i < left, s["free"][(start + i).clamp(max=s["free"].numel() - 1)], s["new_free"])
    place = torch.where(freed, left + freed.cumsum(0) - 1, pages)
    new_free = torch.cat([new_free, new_free[:1]]).scatter(0, place, i.int())[:pages]
    copies = torch.where(copy[:, None], torch.stack([last, fresh], 1), -1)
    return {"new_table": new_table.int(), "new_lens": torch.where(ok & ~none, keep, 0).int(), "new_shares": shares.clamp(min=0).int(),
            "new_free": new_free, "new_span": torch.stack([left * 0, left + freed.sum()]).int(), "copies": copies.int()}


def _plain_copy(s):
    pool, pairs = s["pool"], s["pairs"].long()
    pairs = torch.where(pairs < 0, pool.shape[1] - 1, pairs)  # onto itself: a page that no pair names
    pool[:, pairs[:, 1]] = pool[:, pairs[:, 0]]
    return pool


# ------------------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    if c["op"] == "tree":
        return _exact_tree(prepare(c, seed))
    if c["op"] == "compact" and c["cache"] == "kv":
        return _exact_compact(prepare(c, seed))
    return None  # whole numbers, and bytes that only move


def _e4m3_table():
    """The 256 values of e4m3, from its definition."""
    vals = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        vals.append(-x if byte >> 7 else x)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, in 64 bits; |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    step = torch.where(x.abs() < 8 * step, step / 2, step)  # a log2 that came out one too high
    step = torch.where(x.abs() >= 16 * step, step * 2, step).clamp(min=2.0 ** -9)
    return torch.round(x / step) * step


def _exact_tree(s):
    c = s["case"]
    P, H, D = c["P"], c["Hkv"], c["D"]
    G = c["Hq"] // H
    codes, scales = _views(s["pool"], c)
    values, out, lse = _e4m3_table(), s["out"].double(), s["lse"].double()
    cu, masks = s["cu"].tolist(), _masks(c)
    for b, n in enumerate(s["lens"].tolist()):
        t0, t1 = cu[b], cu[b + 1]
        nq = t1 - t0
        if not nq:
            continue
        front = n - nq
        if n == 0:
            out[t0:t1], lse[t0:t1] = 0.0, -math.inf
            continue
        pos = torch.arange(n, device="cuda")
        page = s["table"][b, pos // P].long()
        shown = torch.tensor([[m >> j & 1 for j in range(nq)] for m in masks[t0:t1]], device="cuda").bool()
        see = torch.cat([shown.new_ones(nq, front), shown], 1)
        if c["k"]:
            listed_keys = torch.zeros(nq, n + 1, dtype=torch.bool, device="cuda")
            at = s["sel"][t0:t1].long()
            listed_keys.scatter_(1, torch.where((at >= 0) & (at < front), at, n), True)
            see[:, :front] = listed_keys[:, :front]
        for h in range(H):
            kv = values[codes[page, h, pos % P].long()] * torch.exp2(scales[page, h, pos % P // BLOCK].double() - 127)[..., None]
            for a in range(0, nq, 16):
                q = s["q"][t0 + a:min(t1, t0 + a + 16), h * G:(h + 1) * G].double()
                x = torch.einsum("rgd,kd->rgk", q, kv[:, 0]) * s["scale"]
                x = torch.where(see[a:a + 16, None], x, -math.inf)
                l = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(l > -math.inf, l, 0.0)[..., None])
                out[t0 + a:t0 + a + q.shape[0], h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", p, kv[:, 1])
                lse[t0 + a:t0 + a + q.shape[0], h * G:(h + 1) * G] = l
    return {"out": out, "lse": lse}


def _exact_compact(s):
    c = s["case"]
    P = c["P"]
    codes, scales = _views(s["pool"], c)
    values = _e4m3_table()[codes.long()]
    exps = scales.int()
    cu, table, paths = s["cu"].tolist(), s["table"].tolist(), s["path"].tolist()
    lens, count = s["lens"].tolist(), s["n_path"].tolist()
    for b in range(c["B"]):
        front = lens[b] - (cu[b + 1] - cu[b])
        at = 0
        while at < count[b]:  # a destination block at a time: what lies behind it is not written yet
            d0 = front + at
            n = min(count[b] - at, BLOCK - d0 % BLOCK)
            to_page, to_blk = table[b][d0 // P], d0 % P // BLOCK
            src = [front + x for x in paths[b][at:at + n]]
            come = [(table[b][x // P], x % P) for x in src]
            top = torch.stack([exps[:, pg, :, t // BLOCK] for pg, t in come]).amax(0)
            held = d0 % BLOCK if at == 0 else 0
            if held:
                top = torch.maximum(top, exps[:, to_page, :, to_blk])
                old = exps[:, to_page, :, to_blk]
                sl = slice(to_blk * BLOCK, to_blk * BLOCK + held)
                values[:, to_page, :, sl] = _round_e4m3(values[:, to_page, :, sl] * torch.exp2((old - top).double())[:, :, None, :, None])
            new = [_round_e4m3(values[:, pg, :, t] * torch.exp2((exps[:, pg, :, t // BLOCK] - top).double())[..., None]) for pg, t in come]
            for x, y in enumerate(new):
                values[:, to_page, :, (d0 + x) % P] = y
            exps[:, to_page, :, to_blk] = top
            at += n
    return {"codes": values, "scales": exps.to(torch.uint8), "lens": None}
