"""The Q8_0 cache on the GPU: write, read and keep against the f64 oracle, bit
for bit (every step of the format is exact or correctly rounded)."""

import numpy as np
import pytest
import torch

import cache_cases as cc
from oracle import cache as oc
from quantized_decode_gemv_q8_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def handle(c):
    return binding.Q8Cache(*(dev(c[n]) for n in ("k", "k_scale", "v", "v_scale")))


def check_cache(cache, c):
    """The whole cache, what no call should have touched among it, bit for bit."""
    torch.cuda.synchronize()
    for n in ("k", "k_scale", "v", "v_scale"):
        got = getattr(cache, n).cpu().numpy()
        assert np.array_equal(got, c[n], equal_nan=n.endswith("scale")), n


def case(seed, lengths, news, heads, dim, page_size, first=0, pad=0):
    rng = np.random.default_rng(seed)
    table, pages = cc.layout(rng, lengths, page_size)
    c = cc.random_cache(rng, pages, heads, page_size, dim)
    offsets = cc.offsets_of(news, first)
    return rng, table, c, offsets, int(offsets[-1]) + pad


# lengths, new tokens, heads, page size: one token; ragged with an empty sequence
# and one whose tokens are all new; a page boundary inside the new tokens;
# more heads than a wave takes at once; more sequences than one search step
SHAPES = [
    ([1], [1], 1, 16),
    ([40, 0, 33, 7], [3, 0, 33, 1], 2, 16),
    ([130, 64], [70, 64], 3, 64),
    ([5, 300], [2, 1], 9, 128),
    ([3] * 70 + [20], [1] * 70 + [17], 1, 16),
    (list(range(1, 131)), [1] * 130, 2, 32),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_write_and_read(shape, dim, dtype):
    lengths, news, heads, page_size = SHAPES[shape]
    rng, table, c, offsets, rows = case((1, shape, dim), lengths, news, heads, dim, page_size)
    k, kf = cc.rows_of(rng, (rows, heads, dim), dtype)
    v, vf = cc.rows_of(rng, (rows, heads, dim), dtype, 30.0)
    cache = handle(c)
    held = (dev(table), dev(np.array(lengths, np.int32)), dev(offsets))
    print(f"[cache] write {shape} dim {dim} {dtype}", flush=True)
    binding.q8_cache_write(cache, k.to(DEV), v.to(DEV), *held)
    oc.write(c, kf, vf, table, lengths, offsets)
    check_cache(cache, c)
    rk, rv = binding.q8_cache_read(cache, *held, rows, dtype=dtype)
    ek, ev = oc.read(c, table, lengths, offsets)
    for got, want in ((rk, ek), (rv, ev)):
        # codes times scales have at most 31 bits, so f64 holds them; one rounding to the type
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(dtype) if dtype == torch.float32
                           else torch.from_numpy((want.astype(np.float32))).to(dtype))


def test_write_special_values():
    """Zeros, ties, the largest and smallest numbers, infinities and NaN."""
    dim, heads = 128, 1
    x = np.zeros((9, heads, dim), np.float32)
    x[1, 0] = np.arange(dim) - 64.0
    x[1, 0, 0], x[1, 0, 32] = 127.0, 63.5           # scales 1 and 1/2: ties among the rest
    x[1, 0, 33:40] = [0.25, 0.75, 1.25, -0.25, -0.75, -1.25, 63.25]
    x[2, 0, :32] = np.float32(1e-45) * np.arange(32)  # the scale underflows, to zero or the smallest number
    x[2, 0, 32:64] = np.float32(1e-45) * 190
    x[2, 0, 64:96] = np.float32(1e-45) * np.arange(100, 132)
    x[2, 0, 96:] = 1e-38 * np.linspace(-1, 1, 32)
    x[3, 0] = 3.4e38 * np.linspace(-1, 1, dim)
    x[4, 0, 5], x[4, 0, 40], x[4, 0, 70] = np.inf, -np.inf, np.nan
    x[4, 0, 100] = -3.0
    x[5, 0, 31], x[5, 0, 32] = np.nan, 7.0
    x[6, 0] = -0.0
    rng = np.random.default_rng(5)
    # values at half steps of their block's scale, and one place beside them
    for r in (7, 8):
        for b in range(4):
            top = np.float32(rng.uniform(0.5, 2.0))
            s = np.float32(np.float64(top) / 127)
            half = ((rng.integers(-126, 126, 32) + 0.5) * np.float64(s)).astype(np.float32)
            if r == 8:
                half = np.nextafter(half, np.float32(np.inf) * rng.choice([-1, 1], 32).astype(np.float32))
            half[0] = top
            x[r, 0, 32 * b:32 * b + 32] = half
    c = cc.random_cache(rng, 2, heads, 16, dim)
    cache = handle(c)
    table, lengths, offsets = np.array([[1]], np.int32), [9], [0, 9]
    held = (dev(table), dev(np.array(lengths, np.int32)), dev(np.array(offsets, np.int32)))
    with np.errstate(all="ignore"):
        oc.write(c, x, x, table, lengths, offsets)
    binding.q8_cache_write(cache, dev(x), dev(x), *held)
    check_cache(cache, c)
    k, _ = binding.q8_cache_read(cache, *held, 9)
    k = k.cpu().numpy()[:, 0]
    assert np.isnan(k[4, :96]).all() and np.isfinite(k[4, 96:]).all()
    assert np.isnan(k[5, :32]).all() and np.isfinite(k[5, 32:]).all()


def test_rows_apart_and_rows_of_no_sequence():
    """Views into a fused projection; rows before and behind the sequences stay as they were."""
    lengths, news, heads, dim = [20, 9], [4, 9], 2, 64
    rng, table, c, offsets, rows = case(7, lengths, news, heads, dim, 16, first=3, pad=2)
    wide, _ = cc.rows_of(rng, (rows, 3 * heads * dim + 8), torch.bfloat16)
    wide = wide.to(DEV)
    k = wide[:, 1:1 + heads * dim].unflatten(1, (heads, dim))                      # not 4-byte aligned
    v = wide[:, heads * dim + 2:2 * heads * dim + 2].unflatten(1, (heads, dim))
    cache = handle(c)
    wide_table = dev(np.concatenate([table, table[::-1]], 1))
    held = (wide_table[:, :table.shape[1]], dev(np.array(lengths, np.int32)), dev(offsets))
    binding.q8_cache_write(cache, k, v, *held)
    oc.write(c, k.float().cpu().numpy(), v.float().cpu().numpy(), table, lengths, offsets)
    check_cache(cache, c)
    out = torch.full((rows, 2 * heads * dim + 1), 5.0, dtype=torch.float16, device=DEV)
    ko = out[:, 1:1 + heads * dim].unflatten(1, (heads, dim))
    vo = out[:, 1 + heads * dim:].unflatten(1, (heads, dim))
    binding.q8_cache_read(cache, *held, rows, k=ko, v=vo)
    ek, ev = oc.read(c, table, lengths, offsets)
    assert np.array_equal(ko[3:-2].cpu().numpy(), ek.astype(np.float16))
    assert np.array_equal(vo[3:-2].cpu().numpy(), ev.astype(np.float16))
    assert bool((out[:3] == 5).all()) and bool((out[-2:] == 5).all()) and bool((out[:, 0] == 5).all())


def bad_descriptions():
    """name, changes to (table, lengths, offsets), rows that are lost (their
    sequences are described wrongly), rows that no longer belong to a sequence."""
    return [
        ("page below", lambda t, n, o: t.__setitem__((1, 0), -1), [4, 5, 6], []),
        ("page above", lambda t, n, o: t.__setitem__((1, 0), 1000), [4, 5, 6], []),
        ("one page of two", lambda t, n, o: t.__setitem__((0, 1), 1 << 30), [2, 3], []),
        ("length too small", lambda t, n, o: n.__setitem__(1, 2), [4, 5, 6], []),
        ("length negative", lambda t, n, o: n.__setitem__(1, -5), [4, 5, 6], []),
        ("length past the table", lambda t, n, o: n.__setitem__(1, 1 << 30), [4, 5, 6], []),
        ("offsets past the rows", lambda t, n, o: o.__setitem__(2, 1 << 30), [], [4, 5, 6]),
        ("offsets descend", lambda t, n, o: o.__setitem__(2, 1), [], [4, 5, 6]),
        ("offsets below", lambda t, n, o: o.__setitem__(0, -1), [], [0, 1, 2, 3]),
    ]


@pytest.mark.parametrize("which", range(len(bad_descriptions())))
def test_bad_descriptions(which):
    """A wrong page, length or offset loses its own tokens and no others."""
    name, change, lost, unowned = bad_descriptions()[which]
    heads, dim, page_size = 2, 128, 16
    rng = np.random.default_rng(11)
    lengths, offsets = np.array([18, 9], np.int32), np.array([0, 4, 7], np.int32)
    table = np.array([[3, 1], [0, -1]], np.int32)
    c = cc.random_cache(rng, 4, heads, page_size, dim)
    k, kf = cc.rows_of(rng, (7, heads, dim), torch.float32)
    fine = {n: x.copy() for n, x in c.items()}
    oc.write(fine, kf, kf, table, lengths, offsets)
    untouched = {n: x.copy() for n, x in c.items()}
    bt, bl, bo = table.copy(), lengths.copy(), offsets.copy()
    change(bt, bl, bo)
    cache = handle(c)
    held = (dev(bt), dev(bl), dev(bo))
    print(f"[cache] {name}", flush=True)
    binding.q8_cache_write(cache, k.to(DEV), k.to(DEV), *held)
    # the lost and the unowned rows' places keep what they held
    want = fine
    for t in lost + unowned:
        b, i = (0, t) if t < 4 else (1, t - 4)
        n = 4 if b == 0 else 3
        page, at = oc.slot_of(table, page_size, b, int(lengths[b]) - n + i)
        for x in want:
            want[x][page, :, at] = untouched[x][page, :, at]
    check_cache(cache, want)
    ko = torch.full((7, heads, dim), 5.0, device=DEV)
    vo = ko.clone()
    binding.q8_cache_read(cache, *held, 7, k=ko, v=vo)
    ek, _ = oc.read(want, table, lengths, offsets)
    got = ko.cpu().numpy()
    for t in range(7):
        if t in lost:
            assert np.isnan(got[t]).all()
        elif t in unowned:
            assert (got[t] == 5).all()
        else:
            assert np.array_equal(got[t], ek[t].astype(np.float32))
    # keep moves nothing of a sequence it cannot place
    binding.q8_cache_keep(cache, *held, dev(np.array([[1, 2], [1, 2]], np.int32)))
    if not lost and not unowned:
        return
    torch.cuda.synchronize()
    b = 0 if lost + unowned and (lost + unowned)[0] < 4 else 1
    other = 1 - b
    moved = {n: x.copy() for n, x in want.items()}
    oc.keep(moved, table, lengths, offsets, [[1, 2] if other == 0 else [], [1, 2] if other == 1 else []])
    pages = [p for p in table[other] if p >= 0]
    for n in moved:
        assert np.array_equal(getattr(cache, n).cpu().numpy()[pages], moved[n][pages]), n


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 8])
def test_keep(heads, dim):
    lengths, news = [100, 1, 64, 0, 45, 90], [70, 1, 64, 0, 20, 33]
    rng, table, c, offsets, _ = case((13, dim, heads), lengths, news, heads, dim, 16)
    kept = [sorted(rng.choice(70, 41, replace=False).tolist()), [0], list(range(64)), [], [19], []]
    width = 66
    keep = np.full((6, width), -1, np.int32)
    for b, x in enumerate(kept):
        keep[b, :len(x)] = x
    keep[4, 1:4] = [19, 25, 26]     # 19 again: the list ends before it
    keep[5, :3] = [33, 0, 1]        # not one of the 33 new tokens: nothing is kept
    keep[3, 0] = 0                  # no new tokens
    cache = handle(c)
    held = (dev(table), dev(np.array(lengths, np.int32)), dev(offsets))
    print(f"[cache] keep dim {dim} heads {heads}", flush=True)
    binding.q8_cache_keep(cache, *held, dev(keep))
    oc.keep(c, table, lengths, offsets, kept)
    check_cache(cache, c)


def test_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32 in the code arrays and whose scales lie
    past 2^31: written, read back and moved, and the same place modulo 2^32 is untouched."""
    heads, page_size, dim = 16, 64, 256
    per_page = heads * page_size * dim
    pages = (1 << 32) // per_page + 40
    cache = binding.Q8Cache.empty(pages, heads, page_size, dim, DEV)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.zero_()
    rng = np.random.default_rng(3)
    high = pages - 3
    low = high - (1 << 32) // per_page
    table = np.array([[5, high]], np.int32)
    lengths, offsets = np.array([80], np.int32), np.array([0, 20], np.int32)
    k, kf = cc.rows_of(rng, (20, heads, dim), torch.float32)
    held = (dev(table), dev(lengths), dev(offsets))
    binding.q8_cache_write(cache, k.to(DEV), k.to(DEV), *held)
    want = {"k": np.zeros((2, heads, page_size, dim), np.int8),
            "k_scale": np.zeros((2, heads, page_size, dim // 32), np.float32)}
    want["v"], want["v_scale"] = want["k"].copy(), want["k_scale"].copy()
    oc.write(want, kf, kf, np.array([[0, 1]]), lengths, offsets)
    for n in want:
        t = getattr(cache, n)
        assert np.array_equal(t[5].cpu().numpy(), want[n][0]) and np.array_equal(t[high].cpu().numpy(), want[n][1])
        assert int(torch.count_nonzero(t[low])) == 0
    rk, rv = binding.q8_cache_read(cache, *held, 20)
    ek, ev = oc.read(want, np.array([[0, 1]]), lengths, offsets)
    assert np.array_equal(rk.cpu().numpy(), ek.astype(np.float32)) and np.array_equal(rv.cpu().numpy(), ev.astype(np.float32))
    binding.q8_cache_keep(cache, *held, dev(np.array([[1, 19]], np.int32)))
    oc.keep(want, np.array([[0, 1]]), lengths, offsets, [[1, 19]])
    for n in want:
        assert np.array_equal(getattr(cache, n)[5].cpu().numpy(), want[n][0])
    # attention over the same pages
    q, qf = cc.rows_of(rng, (20, heads, dim), torch.float32)
    out = binding.q8_cache_attention(q.to(DEV), cache, *held)
    ref, spread, size = oc.attention(qf, want, np.array([[0, 1]]), lengths, offsets, dim ** -0.5)
    assert (np.abs(out.cpu().numpy() - ref) <= cc.attention_bound(ref, spread, size, torch.float32)).all()


def test_more_rows_and_sequences_than_one_launch_takes():
    """2^24 rows are a launch of writes and reads, 2^22 sequences one of keep."""
    rows, page = (1 << 24) + 5, 1024
    pages = -(-rows // page)
    cache = binding.Q8Cache.empty(pages, 1, page, 64, DEV)
    gen = torch.Generator(device=DEV).manual_seed(5)
    k = torch.randn((rows, 1, 64), generator=gen, device=DEV, dtype=torch.float16)
    held = (torch.arange(pages, dtype=torch.int32, device=DEV)[None],
            torch.tensor([rows], dtype=torch.int32, device=DEV), torch.tensor([0, rows], dtype=torch.int32, device=DEV))
    print("[cache] rows past one launch", flush=True)
    binding.q8_cache_write(cache, k, k, *held)
    rk, rv = binding.q8_cache_read(cache, *held, rows, dtype=torch.float16)
    at = torch.cat([torch.arange(8), torch.arange((1 << 24) - 8, rows)])
    kf = k[at.to(DEV)].float().cpu().numpy()
    small = {"k": np.zeros((1, 1, 32, 64), np.int8), "k_scale": np.zeros((1, 1, 32, 2), np.float32)}
    small["v"], small["v_scale"] = small["k"].copy(), small["k_scale"].copy()
    one = (np.array([[0]], np.int32), np.array([len(at)], np.int32), np.array([0, len(at)], np.int32))
    oc.write(small, kf, kf, *one)
    want = torch.from_numpy(oc.read(small, *one)[0].astype(np.float32)).half()
    assert torch.equal(rk[at.to(DEV)].cpu(), want) and torch.equal(rk, rv)
    far = (rk - k).abs().amax().item()  # half a step of the largest block, and f16's rounding of both
    assert far <= float(k.abs().amax()) * (1 / 254 + 2 ** -9)

    seqs = (1 << 22) + 3
    table = torch.zeros((seqs, 1), dtype=torch.int32, device=DEV)
    table[-3:, 0] = torch.arange(1, 4, device=DEV)
    lengths = torch.zeros(seqs, dtype=torch.int32, device=DEV)
    lengths[-3:] = 2
    offsets = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
    offsets[-3:] = torch.tensor([2, 4, 6], device=DEV)
    before = cache.k[:4, 0, :2].clone()
    print("[cache] sequences past one launch", flush=True)
    binding.q8_cache_keep(cache, table, lengths, offsets, torch.ones((seqs, 1), dtype=torch.int32, device=DEV))
    assert torch.equal(cache.k[1:4, 0, 0], before[1:, 1]) and torch.equal(cache.k[1:4, 0, 1], before[1:, 1])
    assert torch.equal(cache.k[0, 0, :2], before[0])


@pytest.mark.parametrize("seqs,where,value", [(4, 2, 1 << 30), (4, 2, -1), (4, 4, 2), (130, 72, 1 << 30), (130, 72, -1),
                                              (130, 71, 1 << 30), (130, 0, -5), (700, 330, -1), (700, 341, 1 << 30)])
def test_a_wrong_offset_loses_only_its_own_sequences(seqs, where, value):
    """Sequences that end past the rows, begin before them or descend have no
    rows; all others keep theirs, in batches of any size."""
    heads, dim, page_size, pad = 1, 64, 16, 3
    rng = np.random.default_rng((17, seqs, where))
    offsets = np.arange(seqs + 1, dtype=np.int32) * 2
    offsets[where] = value
    rows = 2 * seqs + pad
    lengths = np.full(seqs, 20, np.int32)
    table = rng.permutation(2 * seqs).reshape(seqs, 2).astype(np.int32)
    c = cc.random_cache(rng, 2 * seqs, heads, page_size, dim)
    k, kf = cc.rows_of(rng, (rows, heads, dim), torch.float32)
    fine = [b for b in range(seqs) if 0 <= offsets[b] <= offsets[b + 1] <= rows and offsets[b + 1] - offsets[b] == 2]
    assert seqs - 2 <= len(fine) < seqs
    cache = handle(c)
    held = (dev(table), dev(lengths), dev(offsets))
    print(f"[cache] offset {where} of {seqs} is {value}", flush=True)
    binding.q8_cache_write(cache, k.to(DEV), k.to(DEV), *held)
    own = np.zeros(rows, bool)
    for b in fine:
        t = slice(offsets[b], offsets[b + 1])
        oc.write(c, kf[t], kf[t], table[b:b + 1], lengths[:1], [0, 2])
        own[t] = True
    check_cache(cache, c)
    ko = torch.full((rows, heads, dim), 5.0, device=DEV)
    vo = ko.clone()
    binding.q8_cache_read(cache, *held, rows, k=ko, v=vo)
    ko = ko.cpu().numpy()
    for b in fine:
        t = slice(offsets[b], offsets[b + 1])
        assert np.array_equal(ko[t], oc.read(c, table[b:b + 1], lengths[:1], [0, 2])[0].astype(np.float32)), b
    assert bool((ko[~own] == 5).all())


def test_keep_with_offsets_past_the_rows():
    """With the number of rows given, a sequence whose offsets pass it has none, as in a write."""
    rng, table, c, offsets, _ = case(18, [40, 40, 40], [8, 8, 8], 2, 64, 16)
    cache = handle(c)
    held = (dev(table), dev(np.array([40, 40, 40], np.int32)), dev(offsets))
    keep = dev(np.tile(np.array([[2, 5, 7]], np.int32), (3, 1)))
    print("[cache] keep with offsets past the rows", flush=True)
    binding.q8_cache_keep(cache, *held, keep, rows=23)
    oc.keep(c, table, [40, 40, 40], offsets, [[2, 5, 7], [2, 5, 7], []])
    check_cache(cache, c)
    binding.q8_cache_keep(cache, *held, keep, rows=24)
    oc.keep(c, table, [40, 40, 40], offsets, [[2, 5, 7]] * 3)
    check_cache(cache, c)
    binding.q8_cache_keep(cache, *held, keep)
    oc.keep(c, table, [40, 40, 40], offsets, [[2, 5, 7]] * 3)
    check_cache(cache, c)
    binding.q8_cache_keep(cache, *held, keep, rows=0)
    check_cache(cache, c)
    with pytest.raises(binding.Q8Error):
        binding.q8_cache_keep(cache, *held, keep, rows=-1)
