"""f64 reference for the cache in 4-bit floats (test infrastructure only).

Written from the definitions, one row and one head at a time:
  * codes 0 .. 7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6, codes 8 .. 15 for their negatives; a
    scale byte e stands for 2^(e - 127), 255 for NaN.
  * Quantising, per 32 channels x: e = the smallest of 2 .. 252 with max|x| <= 7 * 2^(e - 127)
    (252 where there is none); the code of the number nearest to x / scale, of two equally
    near the even code, with x's sign.  A block that holds an infinity or a NaN: e = 255, codes 0.
  * Storage: channel d = 32 b + 2 j + i is nibble i (low first) of byte j * (dim / 32) + b of a
    key's row; of a value's, of byte (4 j + token % 4) * (dim / 32) + b of the 2 * dim bytes that
    tokens 4 n .. 4 n + 3 of a page share.

A cache here is a dict of numpy u8 arrays k, k_scale, v, v_scale shaped
[pages, heads, page_size, dim / 2 or dim / 32].
"""

import numpy as np

from . import cache as oc

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def byte_of_channel(name, dim, at):
    """(byte within a page's codes of one head, nibble) of every channel of token `at` of the page."""
    byte, nibble = np.empty(dim, np.int64), np.empty(dim, np.int64)
    nb = dim // 32
    for d in range(dim):
        b, j, i = d // 32, d % 32 // 2, d % 2
        if name == "v":
            byte[d] = at // 4 * 2 * dim + (4 * j + at % 4) * nb + b
        else:
            byte[d] = at * (dim // 2) + j * nb + b
        nibble[d] = i
    return byte, nibble


def quantise_row(x):
    """(codes u8 [dim] in natural order, scale bytes [dim / 32]) of one row of f32 values."""
    x = np.asarray(x, np.float32).astype(np.float64)
    codes, scales = np.zeros(x.size, np.uint8), np.zeros(x.size // 32, np.uint8)
    for b in range(x.size // 32):
        blk = x[32 * b:32 * b + 32]
        if not np.isfinite(blk).all():
            scales[b] = 255
            continue
        top = np.abs(blk).max()
        e = next((e for e in range(2, 253) if top <= 7 * 2.0 ** (e - 127)), 252)
        scales[b] = e
        for i, y in enumerate(np.abs(blk) / 2.0 ** (e - 127)):
            far = np.abs(GRID - min(y, 6.0))
            near = [c for c in range(8) if far[c] == far.min()]
            codes[32 * b + i] = near[0] if len(near) == 1 else [c for c in near if c % 2 == 0][0]
            if np.signbit(blk[i]):
                codes[32 * b + i] |= 8
    return codes, scales


def _flat(cache, name, page, head):
    """The bytes of one head of one page."""
    return cache[name][page, head].reshape(-1)


def put(cache, name, page, head, at, codes, scales):
    """Stores one row of natural-order codes."""
    byte, nibble = byte_of_channel(name, codes.size, at)
    flat = _flat(cache, name, page, head)
    low = codes[nibble == 0]
    high = codes[nibble == 1]
    assert np.array_equal(byte[nibble == 0], byte[nibble == 1])
    flat[byte[nibble == 0]] = low | high << 4
    cache[name + "_scale"][page, head, at] = scales


def get(cache, name, page, head, at):
    """(codes in natural order, scales) of one row."""
    dim = 2 * cache[name].shape[3]
    byte, nibble = byte_of_channel(name, dim, at)
    codes = _flat(cache, name, page, head)[byte] >> (4 * nibble).astype(np.uint8) & 15
    return codes, cache[name + "_scale"][page, head, at].copy()


def values(codes, scales):
    """f64 values of natural-order codes [..., dim] and scale bytes [..., dim / 32]."""
    size = np.where(codes >= 8, -1.0, 1.0) * GRID[codes & 7]
    step = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return size * np.repeat(step, 32, axis=-1)


def write(cache, k, v, table, lengths, offsets):
    """Writes rows k, v [rows, heads, dim] (f32 values) into the cache, in place."""
    _, heads, page_size, _ = cache["k"].shape
    for b in range(len(lengths)):
        n = offsets[b + 1] - offsets[b]
        for i in range(n):
            page, at = oc.slot_of(table, page_size, b, lengths[b] - n + i)
            for h in range(heads):
                for name, rows in (("k", k), ("v", v)):
                    put(cache, name, page, h, at, *quantise_row(rows[offsets[b] + i, h]))


def sequence(cache, name, table, b, length):
    """f64 values [heads, length, dim] of sequence b's tokens."""
    pages, heads, page_size, half = cache[name].shape
    dim = 2 * half
    places = np.array([byte_of_channel(name, dim, at) for at in range(page_size)])      # [page, 2, dim]
    own = np.asarray(table[b, :-(-length // page_size)], dtype=np.int64)
    flat = cache[name][own].reshape(own.size, heads, -1)
    codes = flat[:, :, places[:, 0].reshape(-1)].reshape(own.size, heads, page_size, dim)
    codes = codes >> (4 * places[:, 1]).astype(np.uint8) & 15
    x = values(codes, cache[name + "_scale"][own])
    return x.transpose(1, 0, 2, 3).reshape(heads, -1, dim)[:, :length]


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
    _, heads, page_size, _ = cache["k"].shape
    for b in range(len(lengths)):
        first = lengths[b] - (offsets[b + 1] - offsets[b])
        for a, j in enumerate(kept[b]):
            ps, s = oc.slot_of(table, page_size, b, first + j)
            pd, d = oc.slot_of(table, page_size, b, first + a)
            for name in ("k", "v"):
                for h in range(heads):
                    put(cache, name, pd, h, d, *get(cache, name, ps, h, s))


def attention(q, cache, table, lengths, offsets, alpha, trees=None):
    """As that of the Q8_0 cache: (out, spread, size)."""
    return oc.attention(q, cache, table, lengths, offsets, alpha, trees, sequence=sequence)
