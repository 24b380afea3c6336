"""Seeded caches, sequences and trees for the cache tests (random numbers and index plumbing only)."""

import numpy as np
import torch

BITS = {torch.float32: 24, torch.bfloat16: 8, torch.float16: 11}


def layout(rng, lengths, page_size, spare=2, pad_columns=1):
    """A table [seqs, pages] of shuffled pages for the lengths, -1 where none is
    needed, and the number of pages."""
    need = [-(-max(0, n) // page_size) for n in lengths]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(need + [0]) + pad_columns), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def random_cache(rng, pages, heads, page_size, dim):
    """A cache of random codes and scales (values of about unit size)."""
    c = {}
    for name in ("k", "v"):
        c[name] = rng.integers(-127, 128, (pages, heads, page_size, dim), dtype=np.int8)
        c[name + "_scale"] = rng.uniform(0.5 / 73, 1.5 / 73, (pages, heads, page_size, dim // 32)).astype(np.float32)
    return c


def offsets_of(news, first=0):
    return np.concatenate([[first], first + np.cumsum(news)]).astype(np.int32)


def random_tree(rng, n):
    """tree_bits of n drafted tokens: each under a random earlier one or under the context."""
    bits = []
    for j in range(n):
        parent = int(rng.integers(-1, j)) if j else -1
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << j)
    return bits


def tree_words(trees, rows, words, first=0):
    """i64 [rows, words] of the sequences' tree_bits."""
    out = np.zeros((rows, words), np.uint64)
    t = first
    for bits in trees:
        for b in bits:
            for w in range(words):
                out[t, w] = b >> 64 * w & (1 << 64) - 1
            t += 1
    return out.view(np.int64)


def rows_of(rng, shape, dtype, scale=1.0):
    """Random rows of dtype (a CPU tensor) and the f32 values they hold."""
    x = torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dtype)
    return x, x.float().numpy()


def attention_bound(out, spread, size, dtype):
    """How far an output may be from the f64 one, element by element.

    Scores: a block's products are exact and summed in f32 (at most 3 matrix
    operations of 32 terms), then scaled and added: under 110 roundings of at
    most 2^-24 of the terms' size, which as a random walk is under 11 of them;
    with the two roundings of the exponent's argument a score is off by at most
    16 * 2^-24 size, below 1e-6 size, and a weight by that factor.  It shifts the
    numerator and the sum of weights, so it counts twice.
    Weights and sums: the weights' parts drop at most 2^-16 of a term for f16
    rows, nothing for f32; with many rows a weight of f32 rows may be two f16, off
    by at most 2^-21 of itself (below 0.5e-6, which counts where few keys carry the
    weight and the walk below is short), one of bf16 rows one f16, off by at most
    2^-11 of itself; the sum over some thousand keys is a random walk of
    f32 roundings, under 64 * 2^-24 of the terms; exp2 and the joins add a few.
    Last, half a step of the output's type.
    """
    eps = 4e-6 + 2e-6 * size[..., None] + {torch.float32: 0, torch.float16: 2.0 ** -16, torch.bfloat16: 2.0 ** -11}[dtype]
    half = torch.finfo(dtype).eps / 2
    return spread * eps * (1 + half) + half * np.abs(out) + torch.finfo(dtype).smallest_normal * half
