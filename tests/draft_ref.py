"""Plain forms of the drafting step's operators, from their definitions in include/idx.h: whole numbers in Python,
sums in 64 bits."""
from __future__ import annotations

import math

import torch

import attn_ref as ref


# ------------------------------------------------------------------------------ trees

def random_tree(n, generator, fan=4):
    """Parents of n nodes, node 0 the root."""
    return [-1] + [int(torch.randint(max(0, j - fan), j, (1,), generator=generator)) for j in range(1, n)]


def ancestors(parents):
    """For each node the set of nodes that it sees: itself and those that it follows."""
    seen = []
    for j, p in enumerate(parents):
        seen.append({j} | (seen[p] if p >= 0 else set()))
    return seen


def mask_words(sets, words):
    """int64 [rows, words] of sets of nodes."""
    rows = []
    for s in sets:
        row = [0] * words
        for j in s:
            row[j // 64] |= 1 << j % 64
        rows.append([x - (1 << 64) if x >> 63 else x for x in row])
    return torch.tensor(rows, dtype=torch.int64).reshape(len(sets), words)


def keys_of(sets, nq, lens, T, sel=None):
    """int32 [T, most]: the key positions that each row attends, -1 behind; sets: of all rows, sequence after sequence."""
    rows, t = [], 0
    for n, q in zip(lens, nq):
        front = n - q
        for _ in range(q):
            row = list(range(max(front, 0))) if sel is None else [int(x) for x in sel[t] if 0 <= int(x) < front]
            row += [front + j for j in sorted(sets[t]) if j < q and front + j >= 0]
            rows.append(row)
            t += 1
    rows += [[]] * (T - t)
    most = max([len(r) for r in rows] + [1])
    return torch.tensor([r + [-1] * (most - len(r)) for r in rows], dtype=torch.int32).reshape(T, most)


# ------------------------------------------------------------------------------ verification

def clean(x):
    x = x.double()
    return torch.where((x >= 0) & (x < math.inf), x, 0.0)


def verify(target, draft, tokens, parents, coins, last, cu, max_path):
    """CPU tensors of any float type, lists. Returns (path, n_path, tokens) as lists, and how far each draw was
    from the nearest border of its running sums, relative to their sum."""
    paths, counts, outs, near = [], [], [], []
    V = target.shape[1]
    for b in range(len(cu) - 1):
        t0, n = cu[b], cu[b + 1] - cu[b]
        if n == 0:
            paths.append([-1] * max_path), outs.append([-1] * max_path), counts.append(0), near.append(1.0)
            continue
        cur, path, out, c, S, gone = 0, [0], [], 0.0, 1.0, set()
        for j in range(1, n):
            x = tokens[t0 + j]
            if parents[t0 + j] != cur or len(path) == max_path or not 0 <= x < V:
                continue
            p = clean(target[t0 + cur])
            if draft is None:
                px = 0.0 if x in gone else float(p[x])
                yes = coins[t0 + j] * S < px
                if not yes:
                    S, gone = max(S - px, 0.0), gone | {x}
            else:
                q = clean(draft[t0 + cur])
                yes = coins[t0 + j] * float(q[x]) * S < float(p[x]) - c * float(q[x])
                if not yes:
                    c += S
                    S = math.fsum((p - c * q).clamp(min=0).tolist())
            if yes:
                path.append(j)
                out.append(x)
                cur, c, S, gone = j, 0.0, 1.0, set()
        p = clean(target[t0 + cur])
        w = p.clone() if draft is None else (p - c * clean(draft[t0 + cur])).clamp(min=0)
        for x in gone:
            w[x] = 0.0
        if not float(w.sum()) > 0:
            w = p
        sums = w.cumsum(0)
        if float(sums[-1]) > 0:
            r = last[b]
            goal = (r if r >= 0 else 0.0) * float(sums[-1])
            above = (sums > goal).nonzero()
            x = int(above[0]) if len(above) else int((w > 0).nonzero()[-1])
            near.append(float((sums - goal).abs().min() / sums[-1]) if goal > 0 else 1.0)
        else:
            x = -1
            near.append(1.0)
        out.append(x)
        paths.append(path + [-1] * (max_path - len(path)))
        outs.append(out + [-1] * (max_path - len(out)))
        counts.append(len(path))
    return paths, counts, outs, near


# ------------------------------------------------------------------------------ compaction

def moves(path, n_path, lens, cu, b, P, width):
    """Front of sequence b's tree and its accepted nodes; (None, []) where it is left alone. And status bits."""
    n, nq, k = lens[b], cu[b + 1] - cu[b], n_path[b]
    if nq < 0 or n < 0 or n > width * P or not 0 <= k <= nq or k > path.shape[1]:
        return None, [], 0x10
    if n < nq:
        return None, [], 0
    nodes = path[b, :k].tolist()
    if any(x <= (nodes[i - 1] if i else -1) or x >= nq for i, x in enumerate(nodes)):
        return None, [], 0x40
    return n - nq, nodes, 0


def kv_compact(pool, Hkv, P, D, path, n_path, lens, cu, table):
    """The effect on a copy of one layer's pool; new lengths; status."""
    pool = pool.clone()
    codes, scales = ref.kv_views(pool, Hkv, P, D)
    vals = ref.e4m3_values()
    new, status, pages = [], 0, pool.shape[0]

    def value(page, h, tok, side):
        e = min(max(int(scales[page, h, tok // 16, side]), 95), 175)
        return vals[codes[page, h, tok, side].long()], e

    for b in range(len(lens)):
        front, nodes, st = moves(path, n_path, lens, cu, b, P, table.shape[1])
        status |= st
        new.append(max(lens[b], 0) if front is None else front + len(nodes))
        i = 0
        while i < len(nodes):
            d0 = front + i
            n = min(len(nodes) - i, 16 - d0 % 16)
            to, blk = int(table[b, d0 // P]), d0 % P // 16
            come = []
            for x in range(n):
                src = front + nodes[i + x]
                pg = int(table[b, src // P])
                if 0 <= pg < pages and 0 <= to < pages:
                    come.append((x, pg, src % P, nodes[i + x] != i + x))
                else:
                    status |= 0x4
            if any(m for *_, m in come):
                held = d0 % 16 if i == 0 else 0
                for h in range(Hkv):
                    for side in range(2):
                        got = [(x, codes[pg, h, t, side].clone(), *value(pg, h, t, side)) for x, pg, t, _ in come]
                        old = min(max(int(scales[to, h, blk, side]), 95), 175)
                        top = max([e for *_, e in got] + ([old] if held else []))
                        for t in range(held):
                            if top > old:
                                at = codes[to, h, blk * 16 + t, side]
                                at.copy_(shift(at, vals[at.long()], old - top))
                        for x, raw, v, e in got:
                            codes[to, h, (d0 + x) % P, side] = shift(raw, v, e - top) if e < top else raw
                        scales[to, h, blk, side] = top
            i += n
    return pool, new, status


def shift(raw, v, by):
    return torch.where(torch.isnan(v), 0x7F, ref.round_e4m3(v * 2.0 ** by)).to(torch.uint8)


def token_places(dtype, P):
    """[P, bytes]: where a token's bytes lie in a page of the indexer's cache."""
    rows = []
    for s in range(P):
        if dtype == 1:
            at = [s // 8 * 1024 + c * 128 + s % 8 * 16 + i for c in range(8) for i in range(16)] + [128 * P + 4 * s + i for i in range(4)]
        elif P == 128:
            at = [(s // 8 * 4 + c) * 128 + s % 8 * 16 + i for c in range(4) for i in range(16)]
            at += [8192 + s % 32 * 16 + s // 32 * 4 + c for c in range(4)]
        else:
            at = [s // 16 * 1024 + s // 8 % 2 * 512 + c * 128 + s % 8 * 16 + i for c in range(4) for i in range(16)]
            at += [4096 + s % 16 * 16 + s // 16 * 4 + c for c in range(4)]
        rows.append(at)
    return torch.tensor(rows)


def k_compact(pool, dtype, P, path, n_path, lens, cu, table):
    pool = pool.clone()
    at, new, status, pages = token_places(dtype, P), [], 0, pool.shape[0]
    for b in range(len(lens)):
        front, nodes, st = moves(path, n_path, lens, cu, b, P, table.shape[1])
        status |= st
        new.append(max(lens[b], 0) if front is None else front + len(nodes))
        for i, x in enumerate(nodes):
            if x == i:
                continue
            ps, pd = int(table[b, (front + x) // P]), int(table[b, (front + i) // P])
            if 0 <= ps < pages and 0 <= pd < pages:
                pool[pd, at[(front + i) % P]] = pool[ps, at[(front + x) % P]]
            else:
                status |= 0x4
    return pool, new, status


# ------------------------------------------------------------------------------ pages

def pages_update(parent, keep, table, lens, P, new_table, shares, free, span, new_free):
    """Lists throughout. Returns (new_table, new_lens, new_shares, new_free, new_span, copies, status)."""
    B, pages, status = len(lens), len(shares), 0
    width, new_width = len(table[0]) if table else 0, len(new_table[0]) if new_table else 0
    new_table, shares, new_free = [list(r) for r in new_table], list(shares), list(new_free)
    head, tail = span
    if not 0 <= head <= tail <= len(free):
        status |= 0x4
        head = tail = 0

    def add(page, by):
        nonlocal status
        if 0 <= page < pages:
            shares[page] += by
        else:
            status |= 0x4

    held = []
    for i in range(B):
        good = 0 <= lens[i] <= width * P
        status |= 0 if good else 0x10
        held.append(-(-lens[i] // P) if good else -1)
        for j in range(max(held[i], 0)):
            add(table[i][j], -1)
    rows = []
    for p, k in zip(parent, keep):
        if p < 0:
            good, n = k == 0, 0
        else:
            good = p < B and held[p] >= 0 and 0 <= k <= lens[p]
            n = -(-k // P) if good else 0
            good = good and n <= new_width
        status |= 0 if good else 0x10
        rows.append(table[p][:n] if good and n else [])
        for page in rows[-1]:
            add(page, 1)
    last = [r[-1] if r and k % P and 0 <= r[-1] < pages else None for r, k in zip(rows, keep)]
    ends = {}
    for b, page in enumerate(last):
        ends.setdefault(page, []).append(b)
    wants = [page is not None and not (shares[page] + 1 == len(ends[page]) and ends[page][0] == b) for b, page in enumerate(last)]
    new_lens, copies, taken = [], [], 0
    for b, r in enumerate(rows):
        pair = [-1, -1]
        n = keep[b] if r else 0
        if wants[b] and head + taken >= tail:
            status |= 0x20
            for page in r:
                add(page, -1)
            r, n = [], 0
        elif wants[b]:
            own = free[head + taken]
            taken += 1
            status |= 0 if 0 <= own < pages else 0x4
            pair = [last[b], own]
            shares[last[b]] -= 1
            r = r[:-1] + [own]
        new_table[b][:len(r)] = r
        new_lens.append(n)
        copies.append(pair)
    out = free[head + taken:tail]
    for page in range(pages):
        if shares[page] < 0:
            status |= 0x4 if shares[page] < -1 else 0
            shares[page] = 0
            out.append(page)
    out = out[:len(new_free)]
    new_free[:len(out)] = out
    return new_table, new_lens, shares, new_free, [0, len(out)], copies, status
