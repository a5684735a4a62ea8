"""fp64 oracle of the paged key-value cache: append, read, decode attention and
page selection, from their definitions (NumPy; no code shared with the CUDA path).

A cache here is a ``Cache``: page arrays ``[n_pages, Hkv, page_size, D]`` of
fp64 values (the values the stored codes stand for), the codes and scales of an
8-bit cache, and the key bounds.  Page tables and lengths are plain lists.
"""
from __future__ import annotations

import math

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 magnitude code 0 .. 126: 4 exponent bits with
    bias 7, 3 mantissa bits, exponent 0 subnormal (code 127 is the NaN)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def quantise(x: np.ndarray, dtype: str):
    """(codes, values, scales) of rows x [..., D] (fp64 holding bf16 values).

    scale = fp32(max|x| / qmax); code = x / scale to the nearest value of the
    type, ties to even.  The quotient of a bf16 value by an fp32 scale is either
    exactly on a border or further from it than an fp64 rounding error, so fp64
    decides every case as exact arithmetic would.  Rows below 2^-100: zeros,
    scale 0.  Rows with a NaN or an infinity: codes 0, scale NaN.
    """
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        bad = ~np.isfinite(amax)
        scale = np.where(amax < TINY, 0.0, (np.where(bad, 0.0, amax) / QMAX[dtype]).astype(np.float32).astype(np.float64))
        t = np.where(scale[..., None] > 0, x / np.where(scale > 0, scale, 1.0)[..., None], 0.0)
        t = np.where(bad[..., None], 0.0, t)
        if dtype == "int8":
            val = np.rint(t)
            code = val.astype(np.int64) & 255
        else:
            grid = e4m3_values()
            mag = np.abs(t)
            hi = np.minimum(np.searchsorted(grid, mag), 126)
            lo = np.maximum(hi - 1, 0)
            dl, dh = mag - grid[lo], grid[hi] - mag
            c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
            val = grid[c] * np.sign(t)
            code = c | np.where(t < 0, 128, 0)
        scale = np.where(bad, np.nan, scale)
        return code.astype(np.uint8), val * scale[..., None], scale


class Cache:
    """pages of values, codes, scales and bounds; all entries start as `fill`."""

    def __init__(self, n_pages, Hkv, page_size, D, dtype="bf16"):
        self.page_size, self.dtype = page_size, dtype
        shape = (n_pages, Hkv, page_size, D)
        self.value = {w: np.zeros(shape) for w in "kv"}
        self.code = {w: np.zeros(shape, np.uint8) for w in "kv"}
        self.scale = {w: np.zeros(shape[:3]) for w in "kv"}
        self.bounds = np.zeros((n_pages, Hkv, 2, D))


def positions(seq_len: int, new: int):
    return range(seq_len - new, seq_len)


def append(cache: Cache, k, v, table, seq_lens, new_lens):
    """k, v fp64 [B, T, Hkv, D] into the cache, as ra_cache_append does."""
    ps = cache.page_size
    for b, (n, new) in enumerate(zip(seq_lens, new_lens)):
        for i, p in enumerate(positions(n, new)):
            page, row = table[b][p // ps], p % ps
            for w, x in (("k", k), ("v", v)):
                if cache.dtype == "bf16":
                    cache.value[w][page, :, row] = x[b, i]
                else:
                    c, val, s = quantise(x[b, i], cache.dtype)
                    cache.code[w][page, :, row], cache.value[w][page, :, row], cache.scale[w][page, :, row] = c, val, s
            old = cache.bounds[page]
            if row == 0:
                old[:, 0], old[:, 1] = math.inf, -math.inf
            old[:, 0] = np.fmin(old[:, 0], k[b, i])
            old[:, 1] = np.fmax(old[:, 1], k[b, i])


def read(cache: Cache, table, seq_lens, first, T, which="k"):
    """[B, T, Hkv, D]: tokens first .. first + T - 1, zero at and behind the end."""
    ps = cache.page_size
    pages = cache.value[which]
    out = np.zeros((len(seq_lens), T, pages.shape[1], pages.shape[3]))
    for b, n in enumerate(seq_lens):
        for t in range(max(0, min(T, n - first))):
            p = first + t
            out[b, t] = pages[table[b][p // ps], :, p % ps]
    return out


def decode(q, cache: Cache, table, seq_lens, new_lens, causal, selected=None):
    """Attention of the new tokens' queries q fp64 [B, Tq, Hq, D] over the cache
    (or over the pages selected[b][g] of each KV head): out fp64, lse.  Rows that
    are not real or see no key: out 0, lse -inf."""
    B, Tq, Hq, D = q.shape
    Hkv, ps = cache.value["k"].shape[1], cache.page_size
    G = Hq // Hkv
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b, (n, new) in enumerate(zip(seq_lens, new_lens)):
        for g in range(Hkv):
            pages = range(-(-n // ps)) if selected is None else [p for p in selected[b][g] if p >= 0]
            pos = np.array([p * ps + r for p in pages for r in range(ps)], dtype=np.int64)
            pos = pos[pos < n] if len(pos) else pos
            if not len(pos):
                continue
            at = np.array([table[b][p // ps] for p in pos])
            kk, vv = (cache.value[w][at, g, pos % ps] for w in "kv")
            for i, p in enumerate(positions(n, new)):
                see = pos <= p if causal else np.ones(len(pos), bool)
                if not see.any():
                    continue
                s = q[b, i, g * G:(g + 1) * G] @ kk[see].T / math.sqrt(D)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                tot = e.sum(-1, keepdims=True)
                out[b, i, g * G:(g + 1) * G] = (e / tot) @ vv[see]
                lse[b, i, g * G:(g + 1) * G] = (m + np.log(tot))[:, 0]
    return out, lse


def select(q, bounds, page_size, table, seq_lens, new_lens, n_sel):
    """int [B, Hkv, n_sel]: the pages with the highest score, ascending, -1 behind.

    score(b, g, p) = max over the real query rows of KV head g of
    sum_d max(q_d lo_pd, q_d hi_pd); the pages that hold new tokens come before
    all others; of equal scores the lower page comes first.  An infinite bound
    (an infinite key) counts as 2^128, so that 0 times it is 0."""
    bounds = np.clip(bounds, -2.0 ** 128, 2.0 ** 128)
    B, Tq, Hq, D = q.shape
    Hkv, ps = bounds.shape[1], page_size
    G = Hq // Hkv
    sel = np.full((B, Hkv, n_sel), -1, np.int64)
    for b, (n, new) in enumerate(zip(seq_lens, new_lens)):
        count = -(-n // ps)
        for g in range(Hkv):
            score = []
            for p in range(count):
                lo, hi = bounds[table[b][p], g]
                rows = q[b, :new, g * G:(g + 1) * G].reshape(-1, D)
                s = max((math.fsum(np.maximum(r * lo, r * hi)) for r in rows), default=-math.inf)
                score.append((0 if new and p >= (n - new) // ps else 1, -s, p))
            best = sorted(p for _, _, p in sorted(score)[:n_sel])
            sel[b, g, :len(best)] = best
    return sel
