"""Pins of the references for the 4-bit cache, the pages and the rotary
positions, by hand examples and identities (CPU)."""

import math

import numpy as np
import pytest

from oracle import cache as oc
from oracle import mx4, pages, rope


def test_codes_by_hand():
    x = np.zeros(64, np.float32)
    x[:12] = [6, -6, 7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0, 0.26]      # scale 1: ties to the even code
    x[32:36] = [7.5, 1, -1, 0.4]                                              # above 7: scale 2
    codes, scales = mx4.quantise_row(x)
    assert scales.tolist() == [127, 128]
    assert codes[:12].tolist() == [7, 15, 7, 0, 2, 2, 4, 4, 6, 6, 8, 1]
    assert codes[32:36].tolist() == [6, 1, 9, 0]             # 3.75 -> 4, 0.5, -0.5, 0.2 -> 0
    assert mx4.values(codes, scales)[32] == 8.0


@pytest.mark.parametrize("top,e", [(0.0, 2), (1e-45, 2), (7 * 2.0 ** -125, 2), (7.5 * 2.0 ** -125, 3), (1.75, 125), (3.4e38, 252),
                                   (np.nextafter(np.float32(1.75), np.float32(2)), 126), (7.0, 127), (8.0, 128)])
def test_scale_bytes(top, e):
    x = np.zeros(32, np.float32)
    x[7] = -top
    assert mx4.quantise_row(x)[1].tolist() == [e]


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_blocks_that_are_not_finite(bad):
    x = np.ones(64, np.float32)
    x[40] = bad
    codes, scales = mx4.quantise_row(x)
    assert scales.tolist() == [125, 255] and not codes[32:].any()
    v = mx4.values(codes, scales)
    assert np.isfinite(v[:32]).all() and np.isnan(v[32:]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_places_fill_a_page_once(dim):
    for name in ("k", "v"):
        seen = set()
        for at in range(16):
            byte, nibble = mx4.byte_of_channel(name, dim, at)
            seen.update(zip(byte.tolist(), nibble.tolist()))
        assert len(seen) == 16 * dim and max(b for b, _ in seen) == 16 * dim // 2 - 1
    byte, nibble = mx4.byte_of_channel("v", dim, 5)          # the second token of the second four
    d = 32 + 2 * 3 + 1
    assert (byte[d], nibble[d]) == (2 * dim + 13 * (dim // 32) + 1, 1)


def test_put_get_and_sequence_agree():
    rng = np.random.default_rng(0)
    c = {n: rng.integers(0, 256, (3, 2, 16, 32 if not n.endswith("e") else 2), dtype=np.uint8)
         for n in ("k", "k_scale", "v", "v_scale")}
    codes, scales = rng.integers(0, 16, 64, dtype=np.uint8), np.array([100, 130], np.uint8)
    for name in ("k", "v"):
        before = mx4.get(c, name, 2, 1, 6)
        mx4.put(c, name, 2, 1, 7, codes, scales)
        got = mx4.get(c, name, 2, 1, 7)
        assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)
        assert np.array_equal(mx4.get(c, name, 2, 1, 6)[0], before[0])
        table = np.array([[0, 2]], np.int32)
        assert np.array_equal(mx4.sequence(c, name, table, 0, 24)[1, 23], mx4.values(codes, scales))


def test_rounding_is_to_the_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal(256).astype(np.float32)
    codes, scales = mx4.quantise_row(x)
    v = mx4.values(codes, scales)
    step = np.repeat(2.0 ** (scales.astype(float) - 127), 32)
    y = np.abs(x) / step
    half = np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))
    assert (np.abs(v - x) <= half * step).all()


def test_attention_reads_the_cache_it_is_given():
    """A cache of ones: the mean of equal values is the value."""
    c = {"k": np.full((1, 1, 16, 32), 0x22, np.uint8), "k_scale": np.full((1, 1, 16, 2), 127, np.uint8),
         "v": np.full((1, 1, 16, 32), 0x55, np.uint8), "v_scale": np.full((1, 1, 16, 2), 128, np.uint8)}
    out, _, size = mx4.attention(np.ones((1, 1, 64)), c, np.array([[0]], np.int32), [9], [0, 1], 0.5)
    assert (out == 6.0).all() and size[0, 0] == 32.0
    assert oc.attention.__defaults__[-1] is oc.sequence


# ------------------------------------------------------------------ pages

def test_fork_and_resize_by_hand():
    refs, table, lengths = [1, 0, 1, 0, 1, 0], [[4, 0, -1], [2, -1, -1]], [20, 16]
    refs, rows, n = pages.fork(refs, table, lengths, [0, 1, 0, 5], 16, 3)
    assert refs == [3, 0, 2, 0, 3, 0] and n == [20, 16, 20, 0]
    assert rows == [[4, 0, -1], [2, -1, -1], [4, 0, -1], [-1, -1, -1]]
    # child 0's last page is shared and partly filled: replaced; child 1's is full: a new one
    refs, rows, moves, missing = pages.resize(refs, rows, n, [21, 17, 20, 0], 16)
    assert rows == [[4, 1, -1], [2, 3, -1], [4, 0, -1], [-1, -1, -1]]
    assert refs == [2, 1, 2, 1, 3, 0] and moves == [[0, 1]] + [[-1, -1]] * 3 and missing == [0] * 4
    # one page is left: the first that lacks one gets it, the others none; a sequence leaves
    refs, rows, moves, missing = pages.resize(refs, rows, [21, 17, 20, 0], [0, 40, 33, 1], 16)
    assert missing == [0, 0, 1 + 1, 1] and rows[1] == [2, 3, 1] and rows[0] == [-1] * 3
    assert refs == [2, 1, 2, 1, 2, 0]


def test_compact_by_hand():
    refs, rows, moves, used = pages.compact([0, 2, 0, 0, 1, 3, 0], [[5, 1], [4, 5], [1, 0]], [32, 20, 33], 16)
    assert used == 3 and moves == [[4, 0], [5, 2], [-1, -1]]
    assert refs == [1, 2, 3, 0, 0, 0, 0] and rows == [[2, 1], [0, 2], [-1, -1]]


# ------------------------------------------------------------------ rotary positions

def test_rotation_by_hand():
    x = np.array([[[1.0, 0.0, 0.0, 2.0, 9.0]]])
    f = [math.pi / 2, math.pi]
    assert np.allclose(rope.rotate(x, [1], f, True), [[[0, 1, 0, -2, 9]]])
    assert np.allclose(rope.rotate(x, [1], f, False), [[[0, 0, 1, -2, 9]]])      # pairs (0, 2) and (1, 3)
    assert np.allclose(rope.rotate(x, [3], f, True, 2.0), [[[0, -2, 0, -4, 9]]])


def test_rotation_back_and_far_positions():
    rng = np.random.default_rng(2)
    x, f = rng.standard_normal((3, 2, 10)), [1.0, 0.1, 0.003]
    y = rope.rotate(x, [5, -7, 1 << 30], f)
    assert np.allclose(rope.rotate(y, [5, -7, 1 << 30], f, inverse=True), x, atol=1e-12)
    # the angle of a far position: from the sum formulas, by doubling
    a, c, s = 0.1, math.cos(0.1), math.sin(0.1)
    for _ in range(20):
        c, s = c * c - s * s, 2 * c * s
    got = rope.angle(1 << 20, a)
    assert abs(math.cos(got) - c) < 1e-8 and abs(math.sin(got) - s) < 1e-8
