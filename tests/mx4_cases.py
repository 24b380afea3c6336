"""Seeded 4-bit caches and attention calls over them, for the tests on the GPU."""

import numpy as np
import torch

import cache_cases as cc
import test_gpu_attention as ga
from oracle import mx4
from quantized_decode_gemv_q8_amd import binding

DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
dev = ga.dev


def random_cache(rng, pages, heads, page_size, dim):
    """Random codes, scales of 2^-3 .. 1."""
    c = {}
    for name in ("k", "v"):
        c[name] = rng.integers(0, 256, (pages, heads, page_size, dim // 2), dtype=np.uint8)
        c[name + "_scale"] = rng.integers(124, 128, (pages, heads, page_size, dim // 32), dtype=np.uint8)
    return c


def handle(c):
    return binding.Mx4Cache(*(dev(c[n]) for n in ("k", "k_scale", "v", "v_scale")))


def bound(out, spread, size, dtype, lost=0.0):
    """How far an output may be from the f64 one, element by element.

    Scores: products of bf16 parts are exact; a score is a chain of at most 8
    blocks * 3 parts matrix operations of 32 terms, under 24 * 8 roundings of at
    most 2^-24 of the terms' size: as a random walk under 14 of them, below 1e-6 of
    size with the two roundings of the exponent's argument.  A weight is off by that
    factor, which shifts the numerator and the sum of weights, so it counts twice.
    Weights: their parts drop at most 2^-16 of a term for bf16 and f16 rows, nothing for
    f32.  The sum over some thousand keys is a random walk of f32 roundings, under
    64 * 2^-24 of the terms; exp2 and the joins add a few.  Last, half a step of the
    output's type.
    lost: of what falls below f32's normal numbers.  A row's kept maximum is no larger
    than its largest score, whose weight is then 1 or more.  A key's weight
    below 2^-126, a part of a weight below it, and what a sum loses there when it is scaled
    to a larger maximum, are each taken as zero: at most 8 times 2^-126 |V| a key
    (the weight or its 3 parts, and 4 roundings of its sum).  It shows where the keys with
    all the weight hold values of zero, as one code in eight does.
    """
    eps = 4e-6 + 2e-6 * size[..., None] + (0 if dtype == torch.float32 else 2.0 ** -16)
    half = torch.finfo(dtype).eps / 2
    return spread * eps * (1 + half) + half * np.abs(out) + torch.finfo(dtype).smallest_normal * half + lost


class Case(ga.Case):
    """An attention call over a random 4-bit cache."""

    def __init__(self, seed, lengths, news, heads, group, dim, page_size, dtype, **kw):
        super().__init__(seed, lengths, news, heads, group, dim, page_size, dtype, **kw)
        self.c = random_cache(np.random.default_rng((7, len(lengths), dim)), len(self.c["k"]), heads, page_size, dim)

    def run(self, cache=None, **kw):
        return binding.q8_mx4_attention(self.q.to(DEV), cache or handle(self.c), *self.held(), tree=self.bits(),
                                        alpha=self.alpha, **kw)

    def want(self):
        return mx4.attention(self.qf, self.c, self.table, self.lengths, self.offsets, self.alpha, self.trees)

    def check(self, out):
        ref, spread, size = self.want()
        own = slice(int(self.offsets[0]), int(self.offsets[-1]))
        got = out.float().cpu().numpy().astype(np.float64)
        scales = self.c["v_scale"][self.c["v_scale"] < 253]
        lost = 8 * 2.0 ** -126 * int(self.lengths.max()) * 6 * 2.0 ** (int(scales.max()) - 127)
        far = (np.abs(got - ref) / bound(ref, spread, size, self.dtype, lost))[own]
        assert far.size == 0 or far.max() <= 1, f"{far.max():.3f} of the bound at {np.unravel_index(far.argmax(), far.shape)}"
