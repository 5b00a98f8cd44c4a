"""The paged key-value cache and its attention in numpy: test infrastructure, no code shared
with the GPU path.

A cache is a dict of planes (k, v: codes [pages, heads, page, dim]; kd, vd: scales
[pages, heads, page, blocks]) and its format; everything beyond the formats' own f32 and
binary16 roundings is f64.
"""

import numpy as np

from . import e4m3 as E

BLOCK = {"q8_0": 32, "e4m3": 128}


def blocks(dim, fmt):
    return -(-dim // BLOCK[fmt])


def quantize(x, fmt):
    """f32 [..., dim] -> (codes, scales): int8 and binary16, or uint8 bit patterns and f32."""
    x = np.ascontiguousarray(x, np.float32)
    dim = x.shape[-1]
    if fmt == "e4m3":
        q, d = E.quantize(x.reshape(-1, dim))
        return q.reshape(x.shape), d.reshape(*x.shape[:-1], -1)
    b = x.reshape(*x.shape[:-1], dim // 32, 32)
    with np.errstate(all="ignore"):
        d = np.abs(b).max(axis=-1) / np.float32(127)
        t = (b / np.where(d == 0, np.float32(1), d)[..., None]).astype(np.float32).astype(np.float64)
        q = np.where(d[..., None] == 0, 0, np.sign(t) * np.floor(np.abs(t) + 0.5))
        return np.clip(q, -127, 127).astype(np.int8).reshape(x.shape), d.astype(np.float16)


def values(q, d, fmt):
    """Codes and scales -> f64."""
    v = E.decode(q) if fmt == "e4m3" else q.astype(np.float64)
    return v * np.repeat(d.astype(np.float64), BLOCK[fmt], axis=-1)[..., : q.shape[-1]]


def rows(cache, slots, which):
    """The cached values at slots, f64 [rows, heads, dim]; zeros outside the cache."""
    q, d = cache[which], cache[which + "d"]
    page = q.shape[2]
    slots = np.asarray(slots, np.int64)
    inside = (slots >= 0) & (slots < q.shape[0] * page)
    s = np.where(inside, slots, 0)
    return np.where(inside[:, None, None], values(q[s // page, :, s % page], d[s // page, :, s % page], cache["format"]), 0.0)


def attention(q, cache, pages, lengths, scale, window=0):
    """(o, lse, bound): o [batch, q_heads, dim] and lse [batch, q_heads] in f64, and a dict of
    what a rounding of the scores or weights may move: see `moved`."""
    batch, hq, dim = q.shape
    page, heads = cache["k"].shape[2], cache["k"].shape[1]
    group = hq // heads
    o = np.zeros((batch, hq, dim))
    lse = np.full((batch, hq), -np.inf)
    parts = []
    for b in range(batch):
        n = min(max(int(lengths[b]), 0), pages.shape[1] * page)
        first = max(0, n - window) if window else 0
        if n == 0:
            parts.append(None)
            continue
        t = np.arange(first, n)
        slots = pages[b, t // page].astype(np.int64) * page + t % page
        k, v = rows(cache, slots, "k"), rows(cache, slots, "v")
        x = q[b].astype(np.float64).reshape(heads, group, dim)
        s = scale * np.einsum("hgd,thd->hgt", x, k)
        terms = abs(scale) * np.einsum("hgd,thd->hgt", np.abs(x), np.abs(k))
        m = s.max(axis=-1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(axis=-1, keepdims=True)
        p /= total
        o[b] = np.einsum("hgt,thd->hgd", p, v).reshape(hq, dim)
        lse[b] = (m + np.log(total)).reshape(hq)
        parts.append((p, s - m, terms, v))
    return o, lse, parts


def moved(part, each, per_term, per_depth, floor):
    """How far o of one sequence may move, [q_heads, dim], and its lse, [q_heads], where weight t is
    off by `each` + per_term * (its score's sum of |terms|) + per_depth * |s_t - m| of itself, and by
    `floor` of the largest weight times the largest |V|."""
    p, below, terms, v = part
    rel = each + per_term * terms + per_depth * np.abs(below)
    mean = (p * rel).sum(axis=-1)
    a = np.abs(v)
    off = np.einsum("hgt,thd->hgd", p * rel, a) + mean[..., None] * np.einsum("hgt,thd->hgd", p, a)
    off += floor * p.shape[-1] * p.max(axis=-1)[..., None] * a.max(axis=(0, 2))[:, None, None]
    return off.reshape(-1, v.shape[-1]), mean.reshape(-1)
