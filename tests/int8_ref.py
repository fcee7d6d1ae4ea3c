"""Plain implementations in 64 bits of what the calls over an INT8 cache and the page calls do: one Python loop over
pages, rows and heads, written from include/pkv.h."""
from __future__ import annotations

import math

import numpy as np


def least_power_of_two(a: float) -> float:
    """The least power of two s >= 2^-126 with a <= 127 s."""
    e = -126
    while 127.0 * 2.0 ** e < a:
        e += 1
    return 2.0 ** e


def append(codes, scales, k, v, cu, ctx, tables):
    """codes int8 [NB, 2, H, bs, D], scales float32 [NB, 2, H] (both changed in place); k, v float64 [T, H, D]."""
    nb, _, heads, bs, _ = codes.shape
    for b in range(len(ctx)):
        n, done = int(cu[b + 1] - cu[b]), 0
        while done < n:
            pos = int(ctx[b]) + done
            off, count = pos % bs, min(bs - pos % bs, n - done)
            rows = slice(int(cu[b]) + done, int(cu[b]) + done + count)
            done += count
            if not 0 <= pos // bs < tables.shape[1]:
                continue
            page = int(tables[b, pos // bs])
            if not 0 <= page < nb:
                continue
            for i, x in enumerate((k, v)):
                for h in range(heads):
                    y = x[rows, h]
                    old = float(scales[page, i, h]) if off else 0.0
                    old = 0.0 if old < 2.0 ** -126 else old
                    if not np.all(np.isfinite(y)) or not math.isfinite(old):
                        scales[page, i, h] = np.nan
                        codes[page, i, h, off:off + count] = 0
                        continue
                    a = float(np.abs(y).max())
                    new = old if a <= 127.0 * old else least_power_of_two(a)
                    if off and new != old:
                        # np.rint: to nearest even
                        codes[page, i, h, :off] = np.rint(codes[page, i, h, :off].astype(np.float64) * (old / new))
                    codes[page, i, h, off:off + count] = np.rint(y / new) if new > 0 else 0
                    scales[page, i, h] = new


def context(codes, scales, table, length):
    """K and V [2, H, length, D] of a sequence, float64."""
    bs = codes.shape[3]
    pages = [int(p) for p in table[:-(-length // bs)]]
    x = codes[pages].astype(np.float64) * scales[pages].astype(np.float64)[..., None, None]
    return x.transpose(1, 2, 0, 3, 4).reshape(2, codes.shape[2], -1, codes.shape[4])[:, :, :length]


def attention(codes, scales, q, cu, lens, tables, scale, causal=True):
    """(out [T, Hq, D], lse [T, Hq]) of the rows of q (float64); a row that sees nothing: 0 and -inf."""
    heads, d = codes.shape[2], codes.shape[4]
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    group = q.shape[1] // heads
    for b, length in enumerate(lens):
        length, r0, n = int(length), int(cu[b]), int(cu[b + 1] - cu[b])
        if length == 0 or n == 0:
            continue
        with np.errstate(invalid="ignore"):
            kv = context(codes, scales, tables[b], length)
        for h in range(q.shape[1]):
            s = q[r0:r0 + n, h] @ kv[0, h // group].T * scale
            if causal:
                for r in range(n):
                    s[r, length - n + r + 1:] = -np.inf
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            out[r0:r0 + n, h] = p @ kv[1, h // group] / l
            lse[r0:r0 + n, h] = (m + np.log(l))[:, 0]
    return out, lse


def copy_pages(pools, src, dst, rows, bs):
    """pools: (array [NB, ...], axis of the rows or None: one entry a page) pairs, source and destination the same."""
    for i, (s, d) in enumerate(zip(src, dst)):
        n = bs if rows is None else int(rows[i])
        for x, axis in pools:
            if axis is None:
                if n > 0:
                    x[d] = x[s]
            else:
                at = [slice(None)] * (x.ndim - 1)
                at[axis - 1] = slice(0, n)
                x[(d,) + tuple(at)] = x[(s,) + tuple(at)]


def fork(pools, tables, lens, parents, fresh, bs):
    """(tables, lens) of the children; the partly filled last pages copied in pools (see copy_pages)."""
    mb = tables.shape[1]
    out, out_lens = np.full((len(parents), mb), -1, np.int32), np.zeros(len(parents), np.int32)
    for c, p in enumerate(parents):
        n = int(lens[p])
        full, rest = n // bs, n % bs
        out[c, :full] = tables[p, :full]
        out_lens[c] = n
        if rest and fresh[c] < 0:
            out[c, full] = tables[p, full]
        elif full < mb and fresh[c] >= 0:
            out[c, full] = fresh[c]
            if rest:
                copy_pages(pools, [int(tables[p, full])], [int(fresh[c])], [rest], bs)
    return out, out_lens
