"""Plain CPU oracle of the operators between the packed linear layers: the cache held in 4
bits, its plan, attention over it and the norms around a block.

TEST INFRASTRUCTURE ONLY, like the layer's oracle beside it: numpy, loops, 64 bits wherever
the definition does not say otherwise, no code shared with the library.  bf16 values are
carried as the float32 values they stand for.
"""
from __future__ import annotations

import numpy as np


def bf16_round(x):
    """float32 values rounded to the nearest bf16 (ties to even), as float32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, np.asarray(x, np.float32)).astype(np.float32)


# ------------------------------------------------------------------------------ the cache

def kv4_quant(x):
    """Codes, scales and minima of x [..., dim] (16-bit values): the definition in fp32 steps.
    Returns (codes uint8 [..., dim/64, 64], s fp16 [..., dim/64], m fp16 [..., dim/64])."""
    x = np.asarray(x).astype(np.float32)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), np.float32(-65504), np.float32(65504))
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    lo, hi = g.min(-1), g.max(-1)
    m = (lo + np.float32(0)).astype(np.float16)          # -0 becomes 0
    s = ((hi - lo) / np.float32(15)).astype(np.float16)
    s = np.where((s == 0) & (hi > lo), np.float16(2.0 ** -24), s)
    sf, mf = s.astype(np.float32)[..., None], m.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((g - mf) / sf)
    c = np.where(sf == 0, 0, np.clip(c, 0, 15))
    return c.astype(np.uint8), s, m


def kv4_values(codes, s, m):
    """m + s c in 64 bits, [..., dim]."""
    v = m.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * codes
    return v.reshape(*v.shape[:-2], v.shape[-2] * 64)


def kv4_block(cache, page_no, head, page, dim):
    """The four parts of one (page, head) block of a cache [pages, heads, bytes], as views."""
    blk = cache[page_no, head]
    half, par = page * dim // 2, page * dim // 16
    return blk[:half], blk[half:2 * half], blk[2 * half:2 * half + par], blk[2 * half + par:]


def kv4_write(cache, slots, k, v, page):
    """Writes rows k, v [T, heads, dim] to their slots, byte by byte as the layout says."""
    pages, heads, _ = cache.shape
    dim = k.shape[2]
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= pages * page:
            continue
        p, tok = divmod(int(slot), page)
        for h in range(heads):
            kc, vc, kp, vp = kv4_block(cache, p, h, page, dim)
            for part, par, x, is_k in ((kc, kp, k, True), (vc, vp, v, False)):
                c, s, m = kv4_quant(x[t, h])
                c = c.reshape(-1)
                n = 4 * (dim // 64)
                par[tok * n:(tok + 1) * n] = np.concatenate([s, m]).view(np.uint8)
                for ch in range(dim):
                    if is_k:
                        nib = ch % 8
                        at = tok * (dim // 2) + ch % 32 // 8 * (dim // 8) + ch // 32 * 4 + nib // 2
                    else:
                        nib = ch // 16
                        at = (tok // 4 * 16 + ch % 16) * 4 + tok % 4
                        at = at * (dim // 32) + nib // 2
                    old = part[at]
                    part[at] = (old & 0x0F) | (c[ch] << 4) if nib % 2 else (old & 0xF0) | c[ch]


# ------------------------------------------------------------------------------ the plan

def kv_plan(fresh, lens, table, pool, count, page, pages, tokens, fit=False):
    """The plan of a step, request by request; with ``fit`` a request whose rows do not fit is
    refused.  Returns a dict; inputs are not changed."""
    table, pool = table.copy(), pool.copy()
    b_all, width = table.shape
    cap = width * page
    held = [min(max(int(n), 0), cap) for n in lens]
    have = [-(-n // page) for n in held]
    top = min(max(int(count), 0), len(pool))
    for b in range(b_all):
        if fresh[b] < 0:
            for j in range(have[b]):
                if top < len(pool):
                    pool[top] = table[b, j]
                top += 1
    top = min(top, len(pool))
    lens_out, cu, slots, pos, ok = [], [0], [], [], []
    needed = taken = rows = 0
    for b in range(b_all):
        f = int(fresh[b])
        add = max(f, 0)
        cu.append(min(cu[-1] + add, 2 ** 31 - 1))   # saturates
        rows += add
        if f < 0:
            lens_out.append(0)
            ok.append(True)
            continue
        fits = held[b] + add <= cap
        need = -(-(held[b] + add) // page) - have[b] if fits else 0
        good = fits and (need == 0 or needed + need <= top) and not (fit and add and rows > tokens)
        if good and need:
            for j in range(need):
                table[b, have[b] + j] = pool[top - 1 - needed - j]
            taken = needed + need
        needed += need
        ok.append(good)
        lens_out.append(held[b] + add if good else held[b])
    for b in range(b_all):
        first = None
        for i in range(min(max(int(fresh[b]), 0), max(tokens - cu[b], 0))):
            p = held[b] + i
            pg = int(table[b, p // page]) if p < cap else -1
            slot = pg * page + p % page if ok[b] and 0 <= pg < pages else -1
            first = slot if first is None else first
            slots.append(slot if first >= 0 else -1)
            pos.append(p)
    pad = tokens - len(slots)
    i32 = np.int32
    return dict(table=table, pool=pool, lens_out=np.array(lens_out, i32).reshape(-1), cu=np.array(cu, i32),
                slots=np.array(slots + [-1] * pad, i32), pos=np.array(pos + [0] * pad, i32),
                count_out=np.array([top - taken, sum(not x for x in ok)], i32))


# ------------------------------------------------------------------------------ attention

def attention(q, k, v, length, scale, window=0, absent=()):
    """Rows q [n, heads, dim] of one request with `length` tokens, k and v [length, kv heads,
    dim] in 64 bits; tokens in `absent` are not there.  Returns out, lse and, for tolerances,
    the probabilities' mass sum P |v| and the largest sum |q||k| of a seen token."""
    q = np.asarray(q, np.float64)
    n, hq, d = q.shape
    hkv = k.shape[1]
    out, mass = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, size = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i in range(n):
        p = length - n + i
        seen = [t for t in range(max(0, p - window + 1 if window else 0), p + 1) if t not in absent]
        if not seen:
            continue
        for x in range(hq):
            h = x // (hq // hkv)
            kk, vv = k[seen, h], v[seen, h]
            s = scale * (kk @ q[i, x])
            top = s.max()
            e = np.exp(s - top)
            out[i, x] = e @ vv / e.sum()
            mass[i, x] = e @ np.abs(vv) / e.sum()
            lse[i, x] = top + np.log(e.sum())
            size[i, x] = abs(scale) * (np.abs(kk) @ np.abs(q[i, x])).max()
    return out, lse, mass, size


# ------------------------------------------------------------------------------ the norms

def residual_norm(x, res, pre, post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-5):
    """h' and y in 64 bits, and the unsigned size of h's terms (for tolerances)."""
    f = np.float64
    h = alpha * np.asarray(res, f)
    size = np.abs(h)
    if x is not None:
        u = np.asarray(x, f)
        if post is not None:
            u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * np.asarray(post, f)
        if gate is not None:
            u = u * np.asarray(gate, f)
        h = h + beta * u
        size = size + np.abs(beta * u)
    y = None if pre is None else h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(pre, f)
    return h, y, size
