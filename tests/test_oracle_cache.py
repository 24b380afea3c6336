"""Pins of the cache oracle: small cases worked out by hand, and identities."""

import numpy as np
import pytest

from oracle import cache as oc


def test_pair_order_is_a_permutation_with_whole_pairs():
    for dim in (64, 128, 256):
        place = oc.place_of_channel(dim)
        assert sorted(place) == list(range(dim))
        assert (place[1::2] == place[0::2] + 1).all()
    # channels 0, 1 of blocks 0..3 come first at 128
    assert list(oc.place_of_channel(128)[[0, 1, 32, 33, 64, 65, 96, 97, 2, 3]]) == [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]


def test_quantise_by_hand():
    x = np.zeros(64, np.float32)
    x[0], x[1], x[2], x[3] = 127.0, 0.5, 1.5, -2.5   # scale 1: ties go to even
    x[4] = -126.6
    codes, scales = oc.quantise_row(x)
    assert scales.tolist() == [1.0, 0.0]
    assert codes[:5].tolist() == [127, 0, 2, -2, -127]
    assert not codes[32:].any()
    x[33] = np.inf
    x[2] = np.nan
    codes, scales = oc.quantise_row(x)
    assert np.isnan(scales).all() and not codes.any()


def test_quantise_is_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((20, 128)).astype(np.float32)
    for row in x:
        codes, scales = oc.quantise_row(row)
        assert (np.abs(oc.value_of_row(codes, scales) - row) <= np.repeat(scales.astype(np.float64), 32) * 0.5).all()
        assert (np.abs(codes.reshape(-1, 32)).max(1) == 127).all()


def test_write_read_keep_follow_the_pages():
    rng = np.random.default_rng(2)
    c = {"k": np.zeros((4, 2, 16, 64), np.int8), "k_scale": np.zeros((4, 2, 16, 2), np.float32)}
    c["v"], c["v_scale"] = c["k"].copy(), c["k_scale"].copy()
    table, lengths, offsets = np.array([[2, 0], [3, -1]]), [18, 5], [0, 3, 5]
    k, v = (rng.standard_normal((5, 2, 64)).astype(np.float32) for _ in range(2))
    oc.write(c, k, v, table, lengths, offsets)
    # tokens 15, 16, 17 of sequence 0: page 2 place 15, page 0 places 0 and 1
    used = np.abs(c["k"]).sum((1, 3)) > 0
    assert used[2].nonzero()[0].tolist() == [15] and used[0].nonzero()[0].tolist() == [0, 1]
    assert used[3].nonzero()[0].tolist() == [3, 4] and not used[1].any()
    rk, rv = oc.read(c, table, lengths, offsets)
    for t in range(5):
        for h in range(2):
            assert (rk[t, h] == oc.value_of_row(*oc.quantise_row(k[t, h]))).all()
            assert (rv[t, h] == oc.value_of_row(*oc.quantise_row(v[t, h]))).all()
    oc.keep(c, table, lengths, offsets, [[1, 2], [1]])
    nk, _ = oc.read(c, table, lengths, offsets)
    assert (nk == rk[[1, 2, 2, 4, 4]]).all()


def test_attention_by_hand():
    # two tokens, one head: scores 0 and ln 3 give weights 1/4 and 3/4
    c = {"k": np.zeros((1, 1, 16, 64), np.int8), "k_scale": np.ones((1, 1, 16, 2), np.float32)}
    c["v"], c["v_scale"] = c["k"].copy(), c["k_scale"].copy()
    c["k"][0, 0, 1, 0] = 1
    c["v"][0, 0, 0, 0], c["v"][0, 0, 1, 0] = 8, -4
    q = np.zeros((2, 1, 64), np.float32)
    q[:, 0, 0] = 2.0
    out, spread, size = oc.attention(q, c, np.array([[0]]), [2], [0, 2], np.log(3.0) / 2)
    assert out[0, 0, 0] == 8 and out[1, 0, 0] == pytest.approx(-1.0)
    assert spread[1, 0, 0] == pytest.approx(5.0) and size[1, 0] == pytest.approx(np.log(3.0))
    # a tree whose second token sees nothing but itself, and a third that sees nothing
    out, _, _ = oc.attention(np.repeat(q, 2, 0)[:3], c, np.array([[0]]), [3], [0, 3], 1.0, [[0b001, 0b010, 0]])
    assert out[0, 0, 0] == 8 and out[1, 0, 0] == -4 and not out[2].any()


def test_sees():
    assert oc.sees(4, 2).astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert oc.sees(4, 2, [0b10, 0b01]).astype(int).tolist() == [[1, 1, 0, 1], [1, 1, 1, 0]]
