"""Rotary positions on the GPU against exact angles in f64."""

import math

import numpy as np
import pytest
import torch

import cache_cases as cc
from oracle import rope as orope
from quantized_decode_gemv_q8_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bound(x, ref, half_rot, interleaved, amplitude, dtype):
    """The angle is exact to 2^-32 of a turn, 2e-9, and in f32 to 2^-25 of itself (at most pi / 4);
    the series are off by 2e-9 and a few f32 roundings: sine and cosine to 3 * 2^-24.  Times the amplitude
    and the two products with their sum: four roundings more, of terms of at most
    |x| + |y| together.  Last, half a step of the type."""
    size = np.zeros_like(ref)
    for i in range(half_rot):
        m, n = (2 * i, 2 * i + 1) if interleaved else (i, i + half_rot)
        size[..., m] = size[..., n] = abs(amplitude) * (np.abs(x[..., m]) + np.abs(x[..., n]))
    half = torch.finfo(dtype).eps / 2
    return size * 7 * 2.0 ** -24 * (1 + half) + (half * np.abs(ref) if dtype != torch.float32 else 0) + \
        torch.finfo(dtype).smallest_normal * half


def check(x, out, positions, r, freq, inverse=False):
    ref = orope.rotate(x, positions, freq, r.interleaved, r.amplitude, inverse)
    got = out.float().cpu().numpy().astype(np.float64)
    lim = bound(x, ref, len(freq), r.interleaved, r.amplitude, out.dtype)
    far = np.abs(got - ref) / lim
    assert far.max() <= 1, f"{far.max():.2f} of the bound at {np.unravel_index(far.argmax(), far.shape)}"
    assert np.array_equal(got[..., 2 * len(freq):], x[..., 2 * len(freq):])


SHAPES = [(1, 1, 64, 64), (5, 3, 128, 128), (3, 2, 128, 32), (4, 1, 80, 20), (2, 5, 256, 256), (3, 2, 96, 6), (2, 2, 7, 2),
          (2, 1, 4096, 4096), (2, 2, 130, 128), (2, 1, 4096, 2), (65, 1, 2, 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_rotation(shape, interleaved, dtype):
    rows, heads, dim, rot = SHAPES[shape]
    rng = np.random.default_rng((1, shape))
    freq = binding.Rope.frequencies(rot)
    r = binding.Rope(freq, interleaved, 1.0, DEV)
    positions = rng.integers(-10, 200000, rows).tolist()
    x, xf = cc.rows_of(rng, (rows, heads, dim), dtype)
    print(f"[rope] {SHAPES[shape]} {interleaved} {dtype}", flush=True)
    for inverse in (False, True):
        out = binding.q8_rope(x.to(DEV), r, positions=ints(positions), inverse=inverse)
        check(xf, out, positions, r, freq, inverse)
    y = x.to(DEV)
    assert binding.q8_rope(y, r, positions=ints(positions), inverse=True, out=y) is y      # in place
    assert torch.equal(y, out)


# A workgroup per row (more heads than a wave has in flight at once, fewer than 2048 rows) and a wave per row, for
# runs of 8 (of 4 for f32), 4 and 1 pairs; all of the head, and part of it with what is left whole or ragged.
MANY_HEADS = [(3, 40, 128, 128), (5, 33, 128, 128), (2, 90, 24, 24), (3, 90, 96, 24), (2, 90, 97, 40), (2, 9, 80, 40), (3, 90, 6, 6),
              (2, 300, 7, 2), (3, 70, 130, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(MANY_HEADS)))
def test_rotation_of_many_heads(shape, interleaved, dtype):
    rows, heads, dim, rot = MANY_HEADS[shape]
    rng = np.random.default_rng((12, shape))
    freq = binding.Rope.frequencies(rot)
    r = binding.Rope(freq, interleaved, 1.0, DEV)
    positions = rng.integers(-10, 200000, rows).tolist()
    x, xf = cc.rows_of(rng, (rows, heads, dim), dtype)
    print(f"[rope] {MANY_HEADS[shape]} {interleaved} {dtype}", flush=True)
    for inverse in (False, True):
        out = binding.q8_rope(x.to(DEV), r, positions=ints(positions), inverse=inverse)
        check(xf, out, positions, r, freq, inverse)
    y = x.to(DEV)
    assert binding.q8_rope(y, r, positions=ints(positions), inverse=True, out=y) is y      # in place
    assert torch.equal(y, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("place", [False, True])
def test_a_step_of_many_heads_by_sequences(place, dtype):
    """Queries and keys of a decode step with rows of no sequence, a workgroup per row."""
    rng = np.random.default_rng(13)
    lengths, news = [40, 0, 33, 7, 100000], [3, 0, 33, 1, 2]
    offsets = cc.offsets_of(news, 2)
    rows = int(offsets[-1]) + 3
    positions = [n - m + i for n, m in zip(lengths, news) for i in range(m)]
    freq = binding.Rope.frequencies(96)
    r = binding.Rope(freq, True, device=DEV)
    (q, qf), (k, kf) = cc.rows_of(rng, (rows, 64, 128), dtype), cc.rows_of(rng, (rows, 8, 128), dtype)
    xs = q.to(DEV), k.to(DEV)
    outs = xs if place else tuple(torch.full(x.shape, 9.0, dtype=x.dtype, device=DEV) for x in xs)
    got = binding.q8_rope(xs, r, lengths=ints(lengths), offsets=torch.from_numpy(offsets).to(DEV), out=outs)
    own = slice(2, rows - 3)
    for x, x0, out in ((qf, q, got[0]), (kf, k, got[1])):
        check(x[own], out[own], positions, r, freq)
        for part in (slice(0, 2), slice(rows - 3, rows)):
            assert torch.equal(out[part].cpu(), x0[part] if place else torch.full_like(x0[part], 9.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_both_sides_of_few_rows(dtype):
    """2047 rows by a workgroup each, 2048 by a wave each: the same bits."""
    rng = np.random.default_rng(14)
    freq = binding.Rope.frequencies(128)
    r = binding.Rope(freq, device=DEV)
    x = torch.randn((2048, 33, 128), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(dtype)
    p = ints(rng.integers(0, 100000, 2048).tolist())
    many, few = binding.q8_rope(x, r, positions=p), binding.q8_rope(x[:2047], r, positions=p[:2047])
    assert torch.equal(many[:2047], few)
    at = [0, 1, 1000, 2046, 2047]
    check(x[at].float().cpu().numpy(), many[at], p[at].tolist(), r, freq)


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "turns", "index"])
def test_far_positions_and_scalings(scaling):
    """Positions up to the ends of 32 bits; frequencies from whole turns to almost none."""
    rng = np.random.default_rng(2)
    r = binding.Rope.scaled(64, 500000.0, scaling, 8.0, length=8192, device=DEV)
    freq = binding.Rope.frequencies(64, 500000.0, scaling, 8.0, 8192)
    assert r.amplitude == (pytest.approx(0.1 * math.log(8) + 1) if scaling == "index" else 1.0)
    positions = [0, 1, -1, 131071, 1 << 20, 2 ** 31 - 1, -2 ** 31, 123456789]
    x, xf = cc.rows_of(rng, (len(positions), 3, 64), torch.float32)
    check(xf, binding.q8_rope(x.to(DEV), r, positions=ints(positions)), positions, r, freq)
    freq = [0.0, 2 * math.pi, 100.0, -1.0, 1e-12, 3.0, math.pi / 2, math.pi / 4]
    r = binding.Rope(freq, True, -2.5, DEV)
    x, xf = cc.rows_of(rng, (len(positions), 1, 16), torch.float32)
    check(xf, binding.q8_rope(x.to(DEV), r, positions=ints(positions)), positions, r, freq)


def test_back_is_the_gradient_and_the_inverse():
    """<g, R x> = <R' g, x> for any g and x; differences of the turn are the turn of differences; and back again."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for interleaved in (False, True):
        r = binding.Rope.scaled(48, interleaved=interleaved, amplitude=1.7, device=DEV)
        positions = ints([3, 70, 5000, 0])
        x, up, d = (torch.randn((4, 3, 64), generator=g, device=DEV) for _ in range(3))
        y, back = binding.q8_rope(x, r, positions=positions), binding.q8_rope(up, r, positions=positions, inverse=True)
        a, b = (up.double() * y.double()).sum(), (back.double() * x.double()).sum()
        # each of the 768 products is off by at most 7 * 2^-24 of sizes of about 4
        assert abs(a - b) <= 768 * 7 * 2.0 ** -24 * 4
        h = 0.5
        moved = binding.q8_rope(x + h * d, r, positions=positions) - y
        assert ((moved - h * binding.q8_rope(d, r, positions=positions)).abs() <= 3 * 7 * 2.0 ** -24 * 20).all()
        r1 = binding.Rope.scaled(48, interleaved=interleaved, device=DEV)
        y = binding.q8_rope(binding.q8_rope(x, r1, positions=positions), r1, positions=positions, inverse=True)
        assert ((y - x).abs() <= 2 * 7 * 2.0 ** -24 * 10).all()


def test_positions_of_sequences():
    """By lengths and offsets, as the cache takes them; rows of none are left as they were."""
    rng = np.random.default_rng(4)
    lengths, news = [40, 0, 33, 7, 100000], [3, 0, 33, 1, 2]
    offsets = cc.offsets_of(news, 2)
    rows = int(offsets[-1]) + 3
    positions = [n - m + i for n, m in zip(lengths, news) for i in range(m)]
    freq = binding.Rope.frequencies(128)
    r = binding.Rope(freq, device=DEV)
    (q, qf), (k, kf) = cc.rows_of(rng, (rows, 5, 128), torch.bfloat16), cc.rows_of(rng, (rows, 2, 128), torch.bfloat16)
    outs = tuple(torch.full(x.shape, 9.0, dtype=x.dtype, device=DEV) for x in (q, k))
    got = binding.q8_rope((q.to(DEV), k.to(DEV)), r, lengths=ints(lengths), offsets=torch.from_numpy(offsets).to(DEV), out=outs)
    own = slice(2, rows - 3)
    for x, out in ((qf, got[0]), (kf, got[1])):
        check(x[own], out[own], positions, r, freq)
        assert bool((out[:2] == 9).all()) and bool((out[-3:] == 9).all())
    # offsets that descend, or pass the rows, give no rows; a length below the new tokens, positions below zero
    one = torch.full(k.shape, 9.0, dtype=k.dtype, device=DEV)
    binding.q8_rope(k.to(DEV), r, lengths=ints([5, 6, 1]), offsets=ints([4, 2, 1 << 30, 1 << 30]), out=one)
    assert bool((one == 9).all())
    binding.q8_rope(k.to(DEV), r, lengths=ints([1]), offsets=ints([0, 3]), out=one)
    check(kf[:3], one[:3], [-2, -1, 0], r, freq)


def test_many_sequences():
    rng = np.random.default_rng(5)
    news = rng.integers(0, 3, 5000).tolist()
    lengths = [n + int(x) for n, x in zip(news, rng.integers(0, 1000, 5000))]
    positions = [n - m + i for n, m in zip(lengths, news) for i in range(m)]
    freq = binding.Rope.frequencies(8)
    r = binding.Rope(freq, device=DEV)
    x, xf = cc.rows_of(rng, (sum(news), 1, 8), torch.float32)
    out = binding.q8_rope(x.to(DEV), r, lengths=ints(lengths), offsets=torch.from_numpy(cc.offsets_of(news)).to(DEV))
    assert torch.equal(out, binding.q8_rope(x.to(DEV), r, positions=ints(positions)))
    check(xf[:300], out[:300], positions[:300], r, freq)


@pytest.mark.parametrize("dtype", TYPES)
def test_views_of_one_projection_in_place(dtype):
    """Queries and keys as views of a fused projection, at any element, turned in place; what lies between stays."""
    rng = np.random.default_rng(6)
    rows, dim = 7, 64
    wide, wf = cc.rows_of(rng, (rows, 1 + 8 * dim + 3), dtype)
    wide = wide.to(DEV)
    before = wide.clone()
    q, k = wide[:, 1:1 + 4 * dim].unflatten(1, (4, dim)), wide[:, 1 + 4 * dim:1 + 6 * dim].unflatten(1, (2, dim))
    positions = list(range(50, 57))
    freq = binding.Rope.frequencies(48)
    r = binding.Rope(freq, device=DEV)
    binding.q8_rope([q, k], r, positions=ints(positions), out=[q, k])
    check(wf[:, 1:1 + 4 * dim].reshape(rows, 4, dim), q, positions, r, freq)
    check(wf[:, 1 + 4 * dim:1 + 6 * dim].reshape(rows, 2, dim), k, positions, r, freq)
    assert torch.equal(wide[:, 1 + 6 * dim:], before[:, 1 + 6 * dim:]) and torch.equal(wide[:, 0], before[:, 0])


def test_refusals():
    r = binding.Rope.scaled(64, device=DEV)
    x, p = torch.zeros((4, 2, 64), device=DEV), ints([0, 1, 2, 3])
    for kw, what in ((dict(positions=p[:3]), "shape"), (dict(positions=p.long()), "int32"), (dict(positions=p, lengths=p), "pass"),
                     (dict(positions=p, out=x[:, :1]), "shape"), (dict(positions=p, out=x[::1, :, :].half()), "float32"),
                     (dict(positions=p, out=(x, x)), "outputs")):
        with pytest.raises(ValueError, match=what):
            binding.q8_rope(x, r, **kw)
    with pytest.raises(TypeError):
        binding.q8_rope(x, r)
    with pytest.raises(TypeError):
        binding.q8_rope(x, None, positions=p)
    with pytest.raises(ValueError, match="turns 64"):
        binding.q8_rope(x[..., :32].contiguous(), r, positions=p)
    with pytest.raises(ValueError, match="one to|between one"):
        binding.q8_rope([x] * 5, r, positions=p)
    room = torch.zeros((5, 2, 64), device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        binding.q8_rope(room[:4], r, positions=p, out=room[1:])
    with pytest.raises(ValueError, match="overlaps"):
        binding.q8_rope([x, room[:4]], r, positions=p, out=[x, x])
    assert binding.q8_rope(x[:0], r, positions=p[:0]).shape == (0, 2, 64)
    assert binding.q8_rope(x[:, :0], r, positions=p).shape == (4, 0, 64)
    with pytest.raises(ValueError):
        binding.Rope([], device=DEV)
    with pytest.raises(binding.Q8Error):
        binding.Rope([float("nan")], device=DEV)


def test_rows_past_32_bits_and_past_one_launch():
    """Rows whose elements lie past 2^32, and more of them than a grid holds."""
    rng = np.random.default_rng(11)
    freq = binding.Rope.frequencies(64)
    r = binding.Rope(freq, device=DEV)
    x, xf = cc.rows_of(rng, (3, 2, 64), torch.bfloat16)
    wide = (1 << 31) + 64
    room = torch.empty(2 * wide + 128, dtype=torch.bfloat16, device=DEV)
    far, out = room.as_strided((3, 2, 64), (wide, 64, 1)), torch.empty((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    far.copy_(x)
    print("[rope] rows far apart", flush=True)
    binding.q8_rope(far, r, positions=ints([5, -7, 90000]), out=out)
    check(xf, out, [5, -7, 90000], r, freq)
    binding.q8_rope(far, r, positions=ints([5, -7, 90000]), out=far)
    assert torch.equal(far, out)
    del room, far

    rows, few = (1 << 24) + 7, torch.tensor([0, 1, 77, (1 << 24) - 1, 1 << 24, (1 << 24) + 6], device=DEV)
    r = binding.Rope([0.7], device=DEV)
    x = torch.randn((rows, 1, 2), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    p = torch.arange(rows, dtype=torch.int32, device=DEV) - 9
    print("[rope] rows past one launch", flush=True)
    out = binding.q8_rope(x, r, positions=p)
    check(x[few].double().cpu().numpy(), out[few], p[few].tolist(), r, [0.7])
    a = (p.double() * 0.7)[:, None]
    want = torch.cat([x[:, 0, :1] * a.cos() - x[:, 0, 1:] * a.sin(), x[:, 0, :1] * a.sin() + x[:, 0, 1:] * a.cos()], 1)
    # in f64 the angles, up to 2^24, are off by 2^-29 before their sines are taken
    size = x.abs().sum(2).double()
    assert bool(((out[:, 0] - want).abs() <= size * (7 * 2.0 ** -24 + 2.0 ** -28)).all())


def test_captured_and_replayed():
    r = binding.Rope.scaled(128, device=DEV)
    q, k, n = torch.randn((6, 8, 128), device=DEV), torch.randn((6, 2, 128), device=DEV), ints([5, 70, 9])
    offsets, outs = ints([0, 2, 3, 6]), None
    outs = (torch.empty_like(q), torch.empty_like(k))
    binding.q8_rope((q, k), r, lengths=n, offsets=offsets, out=outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.q8_rope((q, k), r, lengths=n, offsets=offsets, out=outs)
    for _ in range(4):
        n += 7
        q.normal_()
        k.normal_()
        want = binding.q8_rope((q, k), r, lengths=n, offsets=offsets)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
