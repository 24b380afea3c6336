"""f64 reference for the Q8_0 cache and the attention over it (test
infrastructure only).

Written from the definitions, one row and one head at a time:
  * Q8_0 of a row, per 32 channels x: scale = f32(max|x| / 127), code = x / scale
    to the nearest whole number, ties to even; a block with an infinity or a
    NaN has scale NaN and codes 0, one whose scale is 0 has codes 0.
  * Storage: the code of channel d = 32 b + 2 j + i is at byte
    j * (dim / 16) + 2 b + i of the row; scale b belongs to block b.
  * Attention: softmax over the tokens a row sees, weights times values; zeros
    for a row that sees nothing.

A cache here is a dict of numpy arrays k, k_scale, v, v_scale shaped
[pages, heads, page_size, dim or dim / 32].
"""

import numpy as np


def place_of_channel(dim):
    """place[d]: byte of channel d in a stored row."""
    place = np.empty(dim, dtype=np.int64)
    for d in range(dim):
        b, j, i = d // 32, d % 32 // 2, d % 2
        place[d] = j * (dim // 16) + 2 * b + i
    return place


def quantise_row(x):
    """(codes i8 [dim] in natural order, scales f32 [dim / 32]) of one row of f32 values."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    codes = np.zeros(x.size, dtype=np.int8)
    scales = np.zeros(x.size // 32, dtype=np.float32)
    for b in range(x.size // 32):
        blk = x[32 * b:32 * b + 32]
        if not np.isfinite(blk).all():
            scales[b] = np.nan
            continue
        s = np.float32(np.abs(blk).max() / 127.0)
        scales[b] = s
        if s > 0:
            codes[32 * b:32 * b + 32] = np.clip(np.rint(blk / np.float64(s)), -127, 127).astype(np.int8)
    return codes, scales


def value_of_row(codes, scales):
    """f64 values of a row of natural-order codes."""
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32)


def slot_of(table, page_size, b, pos):
    return int(table[b, pos // page_size]), pos % page_size


def write(cache, k, v, table, lengths, offsets):
    """Writes rows k, v [rows, heads, dim] (f32 values) into the cache, in place."""
    _, heads, page_size, dim = cache["k"].shape
    place = place_of_channel(dim)
    for b in range(len(lengths)):
        n = offsets[b + 1] - offsets[b]
        for i in range(n):
            page, at = slot_of(table, page_size, b, lengths[b] - n + i)
            for h in range(heads):
                for name, rows in (("k", k), ("v", v)):
                    codes, scales = quantise_row(rows[offsets[b] + i, h])
                    cache[name][page, h, at, place] = codes
                    cache[name + "_scale"][page, h, at] = scales


def sequence(cache, name, table, b, length):
    """f64 values [heads, length, dim] of sequence b's tokens."""
    _, heads, page_size, dim = cache[name].shape
    place = place_of_channel(dim)
    n = -(-length // page_size)
    pages = np.asarray(table[b, :n], dtype=np.int64)
    codes = cache[name][pages].transpose(1, 0, 2, 3).reshape(heads, -1, dim)[:, :length][..., place]
    scales = cache[name + "_scale"][pages].transpose(1, 0, 2, 3).reshape(heads, -1, dim // 32)[:, :length]
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32, axis=-1)


def read(cache, table, lengths, offsets):
    """(k, v) f64 [rows, heads, dim]: the newest tokens of every sequence."""
    out = []
    for name in ("k", "v"):
        parts = []
        for b in range(len(lengths)):
            n = offsets[b + 1] - offsets[b]
            if n:
                parts.append(sequence(cache, name, table, b, lengths[b])[:, lengths[b] - n:].transpose(1, 0, 2))
        out.append(np.concatenate(parts))
    return tuple(out)


def keep(cache, table, lengths, offsets, kept):
    """Moves new token kept[b][a] to the place of new token a, one after another."""
    page_size = cache["k"].shape[2]
    for b in range(len(lengths)):
        first = lengths[b] - (offsets[b + 1] - offsets[b])
        for a, j in enumerate(kept[b]):
            ps, s = slot_of(table, page_size, b, first + j)
            pd, d = slot_of(table, page_size, b, first + a)
            for name in ("k", "k_scale", "v", "v_scale"):
                cache[name][pd, :, d] = cache[name][ps, :, s]


def sees(length, n, tree_bits=None):
    """bool [n, length]: what the n newest of `length` tokens see.  tree_bits:
    one whole number per new token, bit j for new token j; None: causal."""
    m = np.zeros((n, length), dtype=bool)
    m[:, :length - n] = True
    for i in range(n):
        for j in range(n):
            m[i, length - n + j] = j <= i if tree_bits is None else bool(tree_bits[i] >> j & 1)
    return m


def attention(q, cache, table, lengths, offsets, alpha, trees=None, sequence=sequence):
    """(out, spread, size): out f64 [rows, q_heads, dim]; spread f64 of out's shape,
    sum_j w_j |V_j| with the softmax weights w (the size of the terms out is
    made of); size f64 [rows, q_heads], the largest alpha * sum_d |q_d K_jd|
    over the tokens seen (the size of the terms of a score).  trees: per
    sequence the tree_bits of sees().  sequence: how the cache's values are read."""
    q = np.asarray(q, dtype=np.float64)
    heads = cache["k"].shape[1]
    group = q.shape[1] // heads
    out, spread, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(len(lengths)):
        n = offsets[b + 1] - offsets[b]
        if n == 0:
            continue
        K = sequence(cache, "k", table, b, lengths[b])
        V = sequence(cache, "v", table, b, lengths[b])
        seen = sees(lengths[b], n, None if trees is None else trees[b])
        for i in range(n):
            at = np.flatnonzero(seen[i])
            if at.size == 0:
                continue
            for f in range(q.shape[1]):
                x = q[offsets[b] + i, f]
                k, v = K[f // group, at], V[f // group, at]
                z = alpha * (k @ x)
                w = np.exp(z - z.max())
                w /= w.sum()
                out[offsets[b] + i, f] = w @ v
                spread[offsets[b] + i, f] = w @ np.abs(v)
                size[offsets[b] + i, f] = abs(alpha) * (np.abs(k) @ np.abs(x)).max()
    return out, spread, size
