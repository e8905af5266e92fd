"""Plain 64-bit forms of the step metadata, the 8-bit KV store and the paged attention, from their
definitions in include/idx.h, and the error bounds that the attention tests hold the kernels to."""
from __future__ import annotations

import math

import torch

BLOCK, E_MIN, E_MAX = 16, -32, 48


def e4m3_values():
    vals = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        vals.append(-x if byte >> 7 else x)
    return torch.tensor(vals, dtype=torch.float64)


def round_e4m3(x):
    """fp64 -> e4m3 codes (uint8): nearest, ties to even, saturating; NaN is stored as 0."""
    vals = e4m3_values()[:127].to(x.device)  # 0 .. 448, increasing; index = code
    a = torch.nan_to_num(x.abs(), nan=0.0, posinf=1e300).clamp(max=448.0)
    hi = torch.searchsorted(vals, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - vals[lo], vals[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    neg = torch.signbit(x) & ~torch.isnan(x)
    return (code + torch.where(neg, 128, 0)).to(torch.uint8)


def exponent(amax: float) -> int:
    """Least E in [E_MIN, E_MAX] with amax <= 448 * 2^E."""
    E = E_MIN
    while E < E_MAX and amax > 448.0 * 2.0 ** E:
        E += 1
    return E


def kv_views(pool, Hkv, P, D):
    n, stride = pool.shape
    head = 2 * P * D + 16
    return (pool.as_strided((n, Hkv, P, 2, D), (stride, head, 2 * D, D, 1), pool.storage_offset()),
            pool.as_strided((n, Hkv, P // BLOCK, 2), (stride, head, 2, 1), pool.storage_offset() + 2 * P * D))


def store(pool, k, v, slots, P):
    """The store's effect on a copy of `pool` (CPU uint8 [pages, stride]); rows block by block."""
    pool = pool.clone()
    n, Hkv, D = k.shape
    codes, scales = kv_views(pool, Hkv, P, D)
    vals = e4m3_values()
    kv = torch.stack([k, v], 2).double()
    total = pool.shape[0] * P
    r = 0
    while r < n:
        s0 = int(slots[r])
        if s0 < 0 or s0 >= total:
            r += 1
            continue
        if r > 0 and 0 <= int(slots[r - 1]) and int(slots[r - 1]) // BLOCK == s0 // BLOCK:
            r += 1  # a row of a block whose run has ended
            continue
        end = r + 1
        while end < n and int(slots[end]) // BLOCK == s0 // BLOCK and int(slots[end]) > int(slots[end - 1]):
            end += 1
        page, blk, f = s0 // P, s0 % P // BLOCK, s0 % BLOCK
        x = kv[r:end]
        a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(3).amax(0)  # [Hkv, 2]
        for h in range(Hkv):
            for side in range(2):
                E = exponent(float(a[h, side]))
                if f:
                    old = min(max(int(scales[page, h, blk, side]) - 127, E_MIN), E_MAX)
                    E = max(E, old)
                    if E > old:
                        kept = codes[page, h, blk * BLOCK:blk * BLOCK + f, side]
                        x_kept = vals[kept.long()]  # a NaN code, which the store never writes, stays one
                        kept.copy_(torch.where(torch.isnan(x_kept), 0x7F, round_e4m3(x_kept * 2.0 ** (old - E))))
                scales[page, h, blk, side] = E + 127
                at = slots[r:end] % P
                codes[page, h, at, side] = round_e4m3(x[:, h, side] * 2.0 ** -E)
        r = end
    return pool


def step_meta(ctx, new, table, P, longest, free, span, num_pages, cap):
    """Python integers throughout. Returns (table, cu, lens, pos, slots, free_next, status)."""
    B, table, status = len(ctx), [list(r) for r in table], 0
    head, tail = span
    if not 0 <= head <= tail <= len(free):
        status |= 0x4
        head = tail = min(max(head, 0), len(free))
    cu, lens, pos, slots, at, nxt = [0], [], [], [], head, head
    end = 0
    for b in range(B):
        q = max(new[b], 0)
        end += q
        cu.append(min(end, cap))
        rows = cu[-1] - cu[-2]
        ok = ctx[b] >= 0 and new[b] >= 0 and ctx[b] + new[b] <= longest and end <= cap
        if not ok:
            status |= 0x10
        else:
            j0, j1 = -(-ctx[b] // P), -(-(ctx[b] + q) // P)
            if j1 > j0 and at + j1 - j0 > tail:
                ok = False
                status |= 0x20
            else:
                nxt = at + j1 - j0  # where the demand up to the last request that was not refused ends
                table[b][j0:j1] = free[at:at + j1 - j0] if j1 > j0 else []
                if any(not 0 <= p < num_pages for p in table[b][j0:j1]):
                    status |= 0x4
            at += j1 - j0
        lens.append(ctx[b] + q if ok else 0)
        for i in range(rows):
            p = ctx[b] + i if ok else 0
            page = table[b][p // P] if ok else -1
            if ok and not 0 <= page < num_pages:
                status |= 0x4
            pos.append(p)
            slots.append(page * P + p % P if ok and 0 <= page < num_pages else -1)
    pos += [0] * (cap - len(pos))
    slots += [-1] * (cap - len(slots))
    return table, cu, lens, pos, slots, nxt, status


def visible(n, q, causal):
    return [min(max(n - q + i + 1, 0), n) if causal else n for i in range(q)]


def attention(q, pool, P, Hkv, table, lens, cu, causal, scale, sel=None, out_type=None):
    """fp64 outputs and lse of every row of a sequence (NaN where no sequence owns the row), and
    the bounds on |out - exact| and |lse - exact|, element by element.

    Bounds. A logit s = scale * q.k is off by at most ds: the fp32 sum of D exact products (each
    step rounds by 2^-24 of at most S = scale * sum |q_d k_d|; the tensor core may cut instead of
    rounding, 2^-23), the factor's three roundings and u's own (8 * 2^-24 * (|s| + 64 for Ev and
    the shift, in units of ln 2)), and bf16 q below 2^-28 of the row's largest (2^-39 of it). The
    weights follow with a relative 2 * ds + 2^-21 (ex2.approx: 2 ulp), and fp16 rounds them by
    2^-11; below fp16's normal range (largest weight at least 2^7, half a subnormal step 2^-25) by
    2^-32 of the row's largest weighted code (u carries V's block scale, so that is taken over
    p * 2^Ev). Sums over n keys: n * 2^-23
    relative. The output's own rounding is half a step of its type."""
    dev = q.device
    T, Hq, D = q.shape
    G = Hq // Hkv
    codes, scales = kv_views(pool, Hkv, P, D)
    vals = e4m3_values().to(dev)
    half = torch.finfo(out_type or q.dtype).eps / 2
    tiny = torch.finfo(out_type or q.dtype).tiny * half * 2
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=dev)
    otol, ltol = out.clone(), lse.clone()
    for b, n in enumerate(lens):
        t0, t1 = cu[b], cu[b + 1]
        if t1 == t0:
            continue
        vis = torch.tensor(visible(n, t1 - t0, causal), device=dev)
        pos = torch.arange(n, device=dev)
        page = table[b, pos // P].long()
        blk = pos % P // BLOCK
        for h in range(Hkv):
            e = scales[page, h, blk].double() - 127 if n else torch.zeros(0, 2, device=dev, dtype=torch.float64)
            kv = vals[codes[page, h, pos % P].long()] * torch.exp2(e)[..., None] if n else \
                torch.zeros(0, 2, D, dtype=torch.float64, device=dev)
            for t in range(t0, t1):
                x = q[t, h * G:(h + 1) * G].double()
                if sel is None:
                    keys = pos[:int(vis[t - t0])]
                else:
                    keys = sel[t].long()
                    keys = keys[(keys >= 0) & (keys < vis[t - t0])]
                hs = slice(h * G, (h + 1) * G)
                if keys.numel() == 0:
                    out[t, hs], lse[t, hs], otol[t, hs], ltol[t, hs] = 0.0, -math.inf, 0.0, 0.0
                    continue
                k, v, ev = kv[keys, 0], kv[keys, 1], e[keys, 1]
                s = scale * (x @ k.T)
                p = torch.softmax(s, -1)
                out[t, hs] = p @ v
                lse[t, hs] = torch.logsumexp(s, -1)
                N = keys.numel()
                S = scale * (x.abs() @ k.abs().T)
                ds = (D + 2) * 2.0 ** -23 * S + 8 * 2.0 ** -24 * (s.abs() + 64)
                ds = ds + 2.0 ** -39 * scale * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1)
                ds = ds.amax(-1, keepdim=True)
                rel = 2 * ds + 2.0 ** -21 + N * 2.0 ** -23
                top = (p * torch.exp2(ev)).amax(-1, keepdim=True)
                A = p @ v.abs()
                o = out[t, hs]
                otol[t, hs] = (2.0 ** -11 + 2 * rel) * A + N * 2.0 ** -32 * 448.0 * top + half * o.abs() * 1.01 + tiny
                ltol[t, hs] = (ds + N * 2.0 ** -23)[:, 0] + 2.0 ** -22 * (1 + lse[t, hs].abs() + 64)
    return out, lse, otol, ltol
