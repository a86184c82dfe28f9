"""Plain 64-bit implementations of the attention operators, one row at a time
(numpy only), and the error bounds that the fp16 roundings imply.  Only tests
import this module."""
from __future__ import annotations

import numpy as np

HALF_F16 = 2.0 ** -11   # half a step of fp16, relative
TINY_F16 = 2.0 ** -25   # half a step of its subnormals


def tables(rows, rotary, base=10000.0):
    f = base ** (-np.arange(0, rotary, 2, dtype=np.float64) / max(rotary, 1))
    a = np.arange(rows, dtype=np.float64)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def pairs(rotary, interleaved):
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def rotate(x, cos, sin, positions, interleaved, dtype=np.float64):
    """x [tokens, heads, D] rotated; every product and sum rounded to `dtype`."""
    y = x.astype(dtype).copy()
    if cos is None:
        return y
    rotary = 2 * cos.shape[1]
    ia, ib = pairs(rotary, interleaved)
    c, s = (t[positions][:, None].astype(dtype) for t in (cos, sin))
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def norm_rotate(x, w, eps, cos, sin, positions, interleaved):
    """(value, bound on the error of an fp32 evaluation rounded once to fp16)."""
    y = x.astype(np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * w.astype(np.float64)
    z = rotate(y, cos, sin, positions, interleaved)
    # fp32: the sum of up to 128 squares in a tree (8 + 4 steps), its root, the
    # quotient and two products are within 16 roundings of 2^-24 for each of the
    # pair's channels; their products and sum add three
    size = np.abs(y)
    if cos is not None:
        ia, ib = pairs(2 * cos.shape[1], interleaved)
        both = size[..., ia] + size[..., ib]
        size[..., ia], size[..., ib] = both, both
    return z, HALF_F16 * np.abs(z) + 19 * 2.0 ** -24 * size * (1 + HALF_F16) + TINY_F16


def quantise(x, bits):
    """The cache's rule in IEEE fp32 steps: codes int8 [..., D], scales fp32 [...]."""
    top = 7 if bits == 4 else 127
    x = x.astype(np.float32)
    s = (np.abs(x).max(-1) / np.float32(top)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / s[..., None])
    q = np.where(np.isfinite(q), q, 0)
    return np.clip(q, -top, top).astype(np.int8), s


def pack4(codes):
    u = codes.astype(np.uint8) & 15
    return u[..., 0::2] | (u[..., 1::2] << 4)


def unpack4(b):
    n = np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1).astype(np.int8)
    return np.where(n > 7, n - 16, n).astype(np.int8)


def values(cache, scale, bits):
    """Stored rows as float64 values."""
    if bits == 16:
        return cache.astype(np.float64)
    c = unpack4(cache) if bits == 4 else cache
    return c.astype(np.float64) * scale[..., None].astype(np.float64)


def visible(mask, chain_i, n):
    if mask is None:
        return np.arange(n) <= chain_i
    words = mask.astype(np.uint32)
    j = np.arange(n)
    return ((words[j // 32] >> (j % 32).astype(np.uint32)) & 1) > 0


def attention(q, K, V, page_size, table, context, cu, mask, scale, seen_only=False):
    """(out, lse, bound of out, bound of lse) in float64; rows of no sequence are NaN.
    K, V float64 [pages, heads, page_size, D].  seen_only: a row's bound knows the tokens
    that the row sees and no others."""
    q = q.astype(np.float64)
    n_rows, qh, D = q.shape
    heads = K.shape[1]
    G = qh // heads
    out, lse = np.full(q.shape, np.nan), np.full((n_rows, qh), np.nan)
    b_out, b_lse = np.zeros(q.shape), np.zeros((n_rows, qh))
    for b in range(len(context)):
        n = cu[b + 1] - cu[b]
        pos = np.arange(context[b] + n)
        pg = table[b, pos // page_size] if len(pos) else np.zeros(0, int)
        for i in range(n):
            row = cu[b] + i
            see = np.ones(len(pos), bool)
            see[context[b]:] = visible(None if mask is None else mask[row], i, n)
            p_, o_ = pg[see], pos[see] % page_size
            for h in range(qh):
                k, v = K[p_, h // G, o_], V[p_, h // G, o_]
                if not len(k):
                    out[row, h], lse[row, h] = 0, -np.inf
                    continue
                s = scale * (k @ q[row, h])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                p = e / z
                out[row, h], lse[row, h] = p @ v, m + np.log(z)
                # scores: D products summed in fp32, each step at worst cut off
                # (2^-23), then three roundings; 2^x is good to 2^-22
                d = abs(scale) * (np.abs(k) @ np.abs(q[row, h])).max() * (D + 3) * 2.0 ** -23 + 2.0 ** -22
                size = p @ np.abs(v)
                # p: half a step of fp16, its score's error twice (p and the sum),
                # the products' fp32 sums; the result: half a step.  A p far below the
                # largest is a subnormal: carrying 2^10 or more, and the quantised
                # values' scale over a power of two at most four times the largest
                # scale among the sequence's rows, it is off by at most
                # 2^-25 2^-10 4 max|v| a token, over the sum of the e's
                most = np.abs(v if seen_only else V[pg, h // G, pos % page_size]).max()
                b_out[row, h] = (size * (HALF_F16 + 2 * d + (len(s) + 8) * 2.0 ** -23) * (1 + HALF_F16)
                                 + HALF_F16 * np.abs(out[row, h]) + TINY_F16
                                 + len(s) * most * 2.0 ** -33 / z)
                b_lse[row, h] = d + (len(s) + 8) * 2.0 ** -24 + abs(lse[row, h]) * 2.0 ** -22 + abs(m) * 2.0 ** -22
    return out, lse, b_out, b_lse


def tree_mask(n, rng, words=None):
    """Ancestor bits of a random tree of n drafted tokens, uint32 [n, words]."""
    words = words or max(1, -(-n // 32))
    m = np.zeros((n, words), np.uint32)
    for i in range(n):
        parent = int(rng.integers(-1, i)) if i else -1
        if parent >= 0:
            m[i] = m[parent]
        m[i, i // 32] |= np.uint32(1 << (i % 32))
    return m
