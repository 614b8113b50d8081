"""Plain CPU oracle of a decoder layer's operators in 8 bits: the norms of queries and keys with
the rotation by position, the cache in 8 bits and the linear layer with one scale per token and
channel.

TEST INFRASTRUCTURE ONLY, like the oracles beside it: numpy, loops, 64 bits wherever the
definition does not say otherwise, no code shared with the library.  bf16 values are carried as
the float32 values they stand for.
"""
from __future__ import annotations

import functools

import numpy as np

RUN = 16


# ---------------------------------------------------------------------- norm and rotation

def head_norm_rotate(x, pos, inv_freq, norm=None, eps=1e-6, neighbours=False):
    """x [T, heads, dim] in 64 bits normed per head and turned; also the size |a| + |b| of the
    terms of each result (for tolerances)."""
    y = np.asarray(x, np.float64).copy()
    if norm is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    out, size = y.copy(), np.abs(y)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        # the exact product is reduced as a fraction of a turn in extended precision
        t = np.asarray(pos, np.longdouble) * np.longdouble(np.float32(inv_freq[i]))
        t = np.remainder(t, 2 * np.longdouble("3.14159265358979323846264338327950288"))
        c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
        a, b = y[..., p], y[..., q]
        out[..., p], out[..., q] = a * c - b * s, a * s + b * c
        size[..., p] = size[..., q] = np.abs(a) + np.abs(b)
    return out, size


# ------------------------------------------------------------------------------ the cache

def block_bytes(page, dim):
    return 2 * page * dim + -(-(page // 2) // 128) * 128


@functools.lru_cache(maxsize=None)
def run_bytes(part, dim):
    """Places of a run's codes, [16, dim]."""
    return np.array([[code_byte(part, t, ch) for ch in range(dim)] for t in range(RUN)])


def code_byte(part, t, ch):
    """Place of a code in its run."""
    if part == 0:
        return ch // 64 * 1024 + ch // 16 % 4 * 256 + t * 16 + ch % 16
    return ch // 64 * 1024 + t // 4 * 256 + ch % 16 * 16 + ch // 16 % 4 * 4 + t % 4


def run_views(cache, page_no, head, run, page, dim):
    """(codes of a run [bytes], its scale as a one-element float32 view) for keys and values."""
    blk = cache[page_no, head]
    scales = blk[2 * page * dim:2 * page * dim + page // 2].view(np.float32)
    n = RUN * dim
    return [(blk[part * page * dim + run * n:part * page * dim + (run + 1) * n], scales[2 * run + part:2 * run + part + 1])
            for part in range(2)]


def clean(x):
    x = np.asarray(x, np.float32)
    return np.clip(np.where(np.isnan(x), np.float32(0), x), np.float32(-65504), np.float32(65504))


def kv8_write(cache, slots, k, v, page):
    """Writes rows k, v [T, heads, dim] to their slots, run by run as the definition says."""
    pages, heads, _ = cache.shape
    dim = k.shape[2]
    runs = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < pages * page:
            runs.setdefault(int(slot) // RUN, []).append(t)
    for run, rows in runs.items():
        places = [int(slots[t]) % RUN for t in rows]
        p, r = divmod(run, page // RUN)
        for h in range(heads):
            for part, ((codes, scale), x) in enumerate(zip(run_views(cache, p, h, r, page, dim), (k, v))):
                x = clean(x[rows, h])
                held = scale[0]
                old = held if 0 not in places and np.isfinite(held) and held > 0 else np.float32(0)
                new = max(old, np.abs(x).max() / np.float32(127))
                ratio = old / new if new > 0 else np.float32(0)
                at = run_bytes(part, dim)
                c = codes[at].astype(np.float32) - np.float32(128)
                if 0 in places:
                    c = np.zeros_like(c)
                if ratio != 1:
                    c = np.clip(np.rint(c * ratio), -127, 127)
                c[places] = np.clip(np.rint(x / new), -127, 127) if new > 0 else 0
                codes[at] = (c + 128).astype(np.uint8)
                scale[0] = new


def kv8_values(cache, slots, page, dim):
    """(values [2][tokens, heads, dim] of keys and values, their scales [2][tokens, heads]) in 64
    bits of the tokens at these slots."""
    heads = cache.shape[1]
    out, sc = np.zeros((2, len(slots), heads, dim)), np.zeros((2, len(slots), heads))
    ch = np.arange(dim)
    for i, slot in enumerate(slots):
        p, t = divmod(int(slot), page)
        for h in range(heads):
            for part, (codes, scale) in enumerate(run_views(cache, p, h, t // RUN, page, dim)):
                out[part, i, h] = (codes[code_byte(part, t % RUN, ch)].astype(np.float64) - 128) * float(scale[0])
                sc[part, i, h] = scale[0]
    return out, sc


# ----------------------------------------------------------------------- the linear layer

def quant_rows(a):
    """Codes and scales of the rows of a (float32 values), in fp32 steps; a row with a NaN or an
    infinity has a scale of NaN and codes of 0."""
    a = np.asarray(a, np.float32)
    a = np.where(np.isfinite(a).all(1)[:, None], a, np.float32(np.nan))
    s = np.abs(a).max(1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(a / s[:, None])
        q = np.where(s[:, None] > 0, np.clip(q, -127, 127), 0)
    return q.astype(np.int8), s


def gemm_w8a8(aq, sa, w, sw):
    """The product in 64 bits, where its sums of whole numbers are exact."""
    acc = aq.astype(np.float64) @ w.astype(np.float64).T
    return acc * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)
