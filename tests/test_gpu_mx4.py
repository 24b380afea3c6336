"""The cache in 4-bit floats on the GPU: write, read and keep bit for bit, and
the attention over it, against the f64 reference."""

import numpy as np
import pytest
import torch

import cache_cases as cc
from mx4_cases import DEV, TYPES, Case, bound, dev, handle, random_cache
from oracle import cache as oc
from oracle import mx4
from quantized_decode_gemv_q8_amd import binding

pytestmark = pytest.mark.gpu
NAMES = ("k", "k_scale", "v", "v_scale")


def check_cache(cache, c):
    """The whole cache, what no call should have touched among it, bit for bit."""
    torch.cuda.synchronize()
    for n in NAMES:
        assert np.array_equal(getattr(cache, n).cpu().numpy(), c[n]), n


def case(seed, lengths, news, heads, dim, page_size, first=0, pad=0):
    rng = np.random.default_rng(seed)
    table, pages = cc.layout(rng, lengths, page_size)
    c = random_cache(rng, pages, heads, page_size, dim)
    offsets = cc.offsets_of(news, first)
    return rng, table, c, offsets, int(offsets[-1]) + pad


def ints(x):
    return dev(np.array(x, np.int32))


SHAPES = [
    ([1], [1], 1, 16),
    ([40, 0, 33, 7], [3, 0, 33, 1], 2, 16),
    ([130, 64], [70, 64], 3, 64),
    ([5, 300], [2, 1], 9, 128),
    ([3] * 70 + [20], [1] * 70 + [17], 1, 16),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_write_and_read(shape, dim, dtype):
    lengths, news, heads, page_size = SHAPES[shape]
    rng, table, c, offsets, rows = case((1, shape, dim), lengths, news, heads, dim, page_size)
    k, kf = cc.rows_of(rng, (rows, heads, dim), dtype)
    v, vf = cc.rows_of(rng, (rows, heads, dim), dtype, 30.0)
    cache, held = handle(c), (dev(table), ints(lengths), dev(offsets))
    print(f"[mx4] write {shape} dim {dim} {dtype}", flush=True)
    binding.q8_mx4_write(cache, k.to(DEV), v.to(DEV), *held)
    mx4.write(c, kf, vf, table, lengths, offsets)
    check_cache(cache, c)
    for got, want in zip(binding.q8_mx4_read(cache, *held, rows, dtype=dtype), mx4.read(c, table, lengths, offsets)):
        # a value has 2 significant bits: exact in every type at these sizes
        assert torch.equal(got.cpu().double(), torch.from_numpy(want))


def test_write_special_values():
    """Zeros, ties and their neighbours, the largest and smallest numbers, infinities and NaN."""
    dim, rng = 128, np.random.default_rng(5)
    x = np.zeros((12, 1, dim), np.float32)
    x[1, 0, :32] = np.linspace(-6, 6, 32)
    x[1, 0, 32:64] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5] * 4
    x[1, 0, 64:96] = np.nextafter(x[1, 0, 32:64], np.float32(0))
    x[1, 0, 96:] = np.nextafter(x[1, 0, 32:64], np.float32(9))          # the largest passes 7: the next scale
    x[2, 0] = -x[1, 0]
    x[3, 0] = np.float32(1e-45) * np.arange(dim)
    x[4, 0] = np.float32(2.0 ** -126) * np.linspace(0, 20, dim)
    x[5, 0] = 3.4028234e38 * np.linspace(-1, 1, dim)
    x[6, 0, 5], x[6, 0, 40], x[6, 0, 70], x[6, 0, 100] = np.inf, -np.inf, np.nan, -3.0
    x[7, 0, 31], x[7, 0, 32] = np.nan, 7.0
    x[8, 0] = -0.0
    for r in (9, 10, 11):       # every middle between codes at every size, and one place beside it
        for b in range(4):
            s = np.float32(2.0 ** rng.integers(-120, 120))
            y = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], 32).astype(np.float32) * s
            if r > 9:
                y = np.nextafter(y, np.float32(np.inf) if r == 10 else np.float32(0))
            y[0] = 6 * s
            x[r, 0, 32 * b:32 * b + 32] = y * rng.choice([-1, 1], 32)
    c = random_cache(rng, 2, 1, 16, dim)
    cache = handle(c)
    table, lengths, offsets = np.array([[1]], np.int32), [13], [0, 12]
    held = (dev(table), ints(lengths), ints(offsets))
    mx4.write(c, x, x, table, lengths, offsets)
    binding.q8_mx4_write(cache, dev(x), dev(x), *held)
    check_cache(cache, c)
    want = mx4.read(c, table, lengths, offsets)[0]
    for dtype in TYPES:
        for got in binding.q8_mx4_read(cache, *held, 12, dtype=dtype):
            ref = torch.from_numpy(want).to(dtype)              # one rounding; infinities where f16 ends
            assert torch.equal(torch.nan_to_num(got.cpu(), nan=77.0), torch.nan_to_num(ref, nan=77.0))


def test_rows_apart_and_rows_of_no_sequence():
    lengths, news, heads, dim = [20, 9], [4, 9], 2, 64
    rng, table, c, offsets, rows = case(7, lengths, news, heads, dim, 16, first=3, pad=2)
    wide, _ = cc.rows_of(rng, (rows, 3 * heads * dim + 8), torch.bfloat16)
    wide = wide.to(DEV)
    k = wide[:, 1:1 + heads * dim].unflatten(1, (heads, dim))                      # not 4-byte aligned
    v = wide[:, heads * dim + 2:2 * heads * dim + 2].unflatten(1, (heads, dim))
    cache = handle(c)
    held = (dev(np.concatenate([table, table[::-1]], 1))[:, :table.shape[1]], ints(lengths), dev(offsets))
    binding.q8_mx4_write(cache, k, v, *held)
    mx4.write(c, k.float().cpu().numpy(), v.float().cpu().numpy(), table, lengths, offsets)
    check_cache(cache, c)
    out = torch.full((rows, 2 * heads * dim + 1), 5.0, dtype=torch.float16, device=DEV)
    ko = out[:, 1:1 + heads * dim].unflatten(1, (heads, dim))
    vo = out[:, 1 + heads * dim:].unflatten(1, (heads, dim))
    binding.q8_mx4_read(cache, *held, rows, k=ko, v=vo)
    for got, want in zip((ko, vo), mx4.read(c, table, lengths, offsets)):
        assert np.array_equal(got[3:-2].cpu().numpy(), want.astype(np.float16))
    assert bool((out[:3] == 5).all()) and bool((out[-2:] == 5).all()) and bool((out[:, 0] == 5).all())


BAD = [
    ("page below", 0, (1, 0), -1, [4, 5, 6], []),
    ("page above", 0, (1, 0), 4, [4, 5, 6], []),
    ("one page of two", 0, (0, 1), 1 << 30, [2, 3], []),
    ("length too small", 1, 1, 2, [4, 5, 6], []),
    ("length negative", 1, 1, -5, [4, 5, 6], []),
    ("length past the table", 1, 1, 1 << 30, [4, 5, 6], []),
    ("offsets past the rows", 2, 2, 1 << 30, [], [4, 5, 6]),
    ("offsets descend", 2, 2, 1, [], [4, 5, 6]),
    ("offsets below", 2, 0, -1, [], [0, 1, 2, 3]),
]


@pytest.mark.parametrize("which", range(len(BAD)))
def test_bad_descriptions(which):
    """A wrong page, length or offset loses its own tokens and no others."""
    name, where, at, value, lost, unowned = BAD[which]
    heads, dim, page_size = 2, 128, 16
    rng = np.random.default_rng(11)
    lengths, offsets = np.array([18, 9], np.int32), np.array([0, 4, 7], np.int32)
    table = np.array([[3, 1], [0, -1]], np.int32)
    c = random_cache(rng, 4, heads, page_size, dim)
    k, kf = cc.rows_of(rng, (7, heads, dim), torch.float32)
    fine, old = {n: x.copy() for n, x in c.items()}, c
    mx4.write(fine, kf, kf, table, lengths, offsets)
    held = [table.copy(), lengths.copy(), offsets.copy()]
    held[where][at] = value
    held = tuple(dev(x) for x in held)
    cache = handle(c)
    print(f"[mx4] {name}", flush=True)
    binding.q8_mx4_write(cache, k.to(DEV), k.to(DEV), *held)
    for t in lost + unowned:        # their places keep what they held
        b, i = (0, t) if t < 4 else (1, t - 4)
        page, place = oc.slot_of(table, page_size, b, int(lengths[b]) - (4, 3)[b] + i)
        for n in ("k", "v"):
            for h in range(heads):
                mx4.put(fine, n, page, h, place, *mx4.get(old, n, page, h, place))
    check_cache(cache, fine)
    ko = torch.full((7, heads, dim), 5.0, device=DEV)
    vo = ko.clone()
    binding.q8_mx4_read(cache, *held, 7, k=ko, v=vo)
    ek, _ = mx4.read(fine, table, lengths, offsets)
    got = ko.cpu().numpy()
    for t in range(7):
        if t in lost:
            assert np.isnan(got[t]).all()
        elif t in unowned:
            assert (got[t] == 5).all()
        else:
            assert np.array_equal(got[t], ek[t].astype(np.float32))
    before = {n: getattr(cache, n).clone() for n in NAMES}
    binding.q8_mx4_keep(cache, *held, dev(np.array([[-1, -1], [1, 2]], np.int32)), rows=7)
    if lost == [4, 5, 6] or unowned == [4, 5, 6]:       # keep moves nothing of a sequence it cannot place
        assert all(torch.equal(getattr(cache, n), x) for n, x in before.items())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 3])
def test_keep(heads, dim):
    lengths, news = [150, 40, 9, 30], [100, 20, 9, 30]
    rng, table, c, offsets, _ = case((3, heads, dim), lengths, news, heads, dim, 16)
    kept = [sorted(rng.choice(100, 60, replace=False).tolist()), [0, 1, 2], [], [29]]
    keep = np.full((4, 70), -1, np.int32)
    for b, x in enumerate(kept):
        keep[b, :len(x)] = x
    keep[2, :2] = [9, 0]            # not below n: ends the list
    keep[1, 3:5] = [2, 7]           # does not ascend: ends the list
    cache = handle(c)
    binding.q8_mx4_keep(cache, dev(table), ints(lengths), dev(offsets), dev(keep))
    mx4.keep(c, table, lengths, offsets, kept)
    check_cache(cache, c)


# ------------------------------------------------------------------ attention

LENGTHS = [
    ([1], [1]),
    ([31, 32, 33, 127, 128, 129], [1, 1, 1, 1, 1, 1]),
    ([40, 0, 333, 7, 90], [3, 0, 33, 1, 0]),
    ([150, 64], [70, 64]),
    ([1500], [2]),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("which", range(len(LENGTHS)))
def test_attention(which, tree, dim, dtype):
    lengths, news = LENGTHS[which]
    heads, group, page = [(1, 1, 16), (2, 4, 64), (3, 7, 16), (1, 5, 128), (2, 8, 32)][which]
    c = Case((21, which, dim, tree), lengths, news, heads, group, dim, page, dtype, tree=tree)
    print(f"[mx4] attention {which} tree {tree} dim {dim} {dtype}", flush=True)
    c.check(c.run())


@pytest.mark.parametrize("group", [1, 2, 3, 16, 17, 31, 33, 40, 64])
def test_groups(group):
    """Groups that fill an item, leave rows over, or are cut into sub-groups."""
    for dim, news in ((128, [1, 1]), (128, [9, 2]), (256, [5, 1])):
        c = Case((22, group, dim), [70, 200], news, 2, group, dim, 16, torch.float32, tree=group % 2 == 0)
        c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_items_of_all_sizes(tree, dim, dtype):
    """On both sides of every number of rows at which an item's size or kernel changes."""
    for n in (16, 17, 32, 33, 64, 65, 96, 97, 128, 129, 257):
        c = Case((48, n, dim), [n + 75, 2 * n], [n, n], 2 if n < 100 else 1, 1, dim, 32, dtype, tree=tree)
        c.check(c.run())
    for group, news in ((7, [14, 13]), (24, [4, 4]), (100, [1, 1]), (130, [1, 1])):
        c = Case((49, group, dim), [190, 33], news, 1, group, dim, 16, dtype, tree=tree)
        c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
def test_many_sequences_and_long_ones(dtype):
    """More sequences than a workgroup has threads; few rows split over many workgroups; a wide tree."""
    rng = np.random.default_rng(23)
    news = rng.integers(0, 3, 300).tolist()
    lengths = [n + int(x) if n else 0 for n, x in zip(news, rng.integers(0, 200, 300))]
    c = Case(23, lengths, news, 2, 2, 64, 16, dtype)
    c.check(c.run())
    c = Case(24, [9000, 3001], [1, 2], 2, 4, 128, 64, dtype)
    c.check(c.run())
    c = Case(25, [700, 1200], [300, 129], 2, 3, 64, 32, dtype)
    c.check(c.run())
    c = Case(26, [400, 90, 70], [200, 3, 70], 2, 4, 128, 64, dtype, tree=True)
    c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 12, 40])
def test_scales_of_all_sizes(news, dim, dtype):
    """Value scales from 2^-40 to 2^40 and key scales of 2^-10 to 1, token by token and block by block."""
    c = Case((27, dim, news), [300], [news], 1, 4, dim, 16, dtype)
    rng = np.random.default_rng(28)
    c.c["v_scale"] = rng.integers(87, 168, c.c["v_scale"].shape).astype(np.uint8)
    c.c["k_scale"] = rng.integers(117, 128, c.c["k_scale"].shape).astype(np.uint8)
    if dtype == torch.float16:      # below 65504
        c.c["v_scale"] = rng.integers(115, 139, c.c["v_scale"].shape).astype(np.uint8)
    c.check(c.run())


def mark_lost(c, name, seq, pos, block, page_size):
    page, at = oc.slot_of(c.table, page_size, seq, pos)
    c.c[name + "_scale"][page, :, at, block] = 255


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [[4, 6], [40, 60], [25, 30]])
def test_lost_values_and_keys(news, dtype):
    """A value scale of 255 loses its block of the rows that see it, a key scale the rows, and no others."""
    c = Case((46, news[0]), [300, 30 + news[1]], news, 1, 4, 128, 64, dtype, tree=True)
    want = c.run().cpu()
    for seq, pos, block in ((0, 5, 2), (1, 30 + 2, 0), (1, 30 + 4, 3)):
        mark_lost(c, "v", seq, pos, block, 64)
    mark_lost(c, "k", 1, 30 + 3, 1, 64)
    out, (ref, spread, size) = c.run().float().cpu().numpy(), c.want()
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    fine = ~np.isnan(ref)
    assert fine.any() and not fine.all()
    assert (np.abs(out - ref)[fine] <= bound(ref, spread, size, dtype)[fine]).all()
    assert np.array_equal(out[fine], want.float().numpy()[fine])


@pytest.mark.parametrize("dtype", TYPES)
def test_what_is_not_seen_changes_nothing(dtype):
    """Behind the last token, and of a draft that no row sees: any bits."""
    for news in ([2, 3], [40, 60], [25, 30]):
        c = Case((45, news[0]), [300, 90], news, 1, 4, 128, 64, dtype, tree=True)
        c.trees[1] = [b & ~(1 << 1) for b in c.trees[1]]
        want = c.run()
        page, at = oc.slot_of(c.table, 64, 1, 90 - news[1] + 1)
        for value in (0, 1, 90, 252, 253, 254, 255):
            c.c["v_scale"][page, :, at] = value
            c.c["k_scale"][page, :, at] = value
            for b, n in enumerate(c.lengths):
                p, a = oc.slot_of(c.table, 64, b, int(n))
                c.c["v_scale"][p, :, a:] = value
                c.c["k_scale"][p, :, a:] = value
            assert torch.equal(c.run(), want), value


def test_rows_that_see_nothing():
    c = Case(27, [5, 40, 3], [5, 3, 3], 2, 2, 128, 16, torch.float32, tree=True)
    c.trees[0][1] = 0
    c.trees[1][0] = 0
    c.trees[2] = [0, 0, 0]
    for alpha in (c.alpha, 0.0, -1.0):
        c.alpha = alpha
        out = c.run()
        c.check(out)
        assert out[1].abs().max() == 0 and out[8:].abs().max() == 0
    none = binding.q8_mx4_attention(c.q.to(DEV), handle(c.c), *c.held(),
                                    tree=torch.zeros((c.rows, 0), dtype=torch.int64, device=DEV))
    assert bool((none[:5] == 0).all()) and bool((none[8:] == 0).all()) and bool((none[5:8] != 0).any())


def test_rows_of_no_sequence_and_queries_apart():
    c = Case(29, [50, 20], [3, 4], 2, 3, 64, 16, torch.float16, first=2, pad=3)
    width = 6 * 64
    wide = torch.zeros((c.rows, width + 9), dtype=torch.float16, device=DEV)
    q = wide[:, 3:3 + width].unflatten(1, (6, 64))
    q.copy_(c.q)
    room = torch.full((c.rows, width + 5), 7.0, dtype=torch.float16, device=DEV)
    out = room[:, 1:1 + width].unflatten(1, (6, 64))
    assert binding.q8_mx4_attention(q, handle(c.c), *c.held(), alpha=c.alpha, out=out) is out
    c.check(out)
    assert bool((room[:2] == 7).all()) and bool((room[-3:] == 7).all())
    assert bool((room[:, 0] == 7).all()) and bool((room[:, 1 + width:] == 7).all())


@pytest.mark.parametrize("news", [[2, 1], [70, 1]])
@pytest.mark.parametrize("alpha", [0.0, -0.3, 1.0, 1e-40])
def test_alpha(alpha, news):
    c = Case(30, [300, 5], news, 1, 4, 128, 16, torch.float32, alpha=alpha)
    c.check(c.run())


def test_large_scores_and_queries():
    for news in ([1, 2], [60, 2], [120, 2], [150, 2]):
        c = Case(31, [500, 77], news, 2, 2, 64, 16, torch.float32, q_scale=60.0)
        c.check(c.run())
        c = Case(32, [500], [news[0]], 2, 2, 64, 16, torch.float32, q_scale=1e30, alpha=1e-31)
        c.check(c.run())
        c = Case(33, [500], [news[0]], 2, 2, 64, 16, torch.float32, q_scale=1e-42)
        c.check(c.run())


@pytest.mark.parametrize("dtype", TYPES)
def test_infinite_and_nan_queries(dtype):
    """A row whose query is not finite gives NaN; its neighbours are as without it."""
    for news in ([4, 1], [70, 1], [60, 1]):
        c = Case(33, [80, 40], news, 1, 4, 128, 16, dtype)
        cache = handle(c.c)
        want = c.run(cache)
        c.q[1, 2, 5] = float("nan")
        c.q[3, 0, 100] = float("inf")
        got = c.run(cache)
        hit = torch.zeros(got.shape[:2], dtype=torch.bool)
        hit[1, 2] = hit[3, 0] = True
        assert bool(torch.isnan(got.cpu()[hit]).all()) and torch.equal(got.cpu()[~hit], want.cpu()[~hit])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [[2, 3, 1], [70, 130, 1], [60, 110, 1]])
def test_attention_over_bad_descriptions(news, dtype):
    c = Case((44, news[0]), [90, 300, 64], news, 2, 2, 64, 16, dtype)
    cache, q = handle(c.c), c.q.to(DEV)
    want = c.run(cache).cpu()
    c.check(want)
    a, b = news[0], news[0] + news[1]
    for name, where, at, value in (("page below", 0, 4, -1), ("page above", 0, 4, len(c.c["k"])), ("page far above", 0, 12, 2 ** 31 - 1),
                                   ("length below its new tokens", 1, 1, news[1] - 1), ("length past the table", 1, 1, 2 ** 31 - 1),
                                   ("offset", 2, 2, 2 ** 30)):
        held = [c.table.copy(), c.lengths.copy(), c.offsets.copy()]
        held[where][(1, at) if where == 0 else at] = value
        print(f"[mx4] {name} {dtype}", flush=True)
        out = torch.full(q.shape, 5.0, device=DEV, dtype=dtype)
        got = binding.q8_mx4_attention(q, cache, *(dev(x) for x in held), alpha=c.alpha, out=out).cpu()
        assert torch.equal(got[:a], want[:a])
        if where == 2:
            assert bool((got[a:] == 5).all())
        else:       # of a wrong page, the rows that see any of its tokens
            first = max(a, a + 16 * at - (300 - news[1])) if where == 0 else a
            assert torch.equal(got[a:first], want[a:first])
            assert bool(torch.isnan(got[first:b]).all()) and torch.equal(got[b], want[b])


@pytest.mark.parametrize("news", [[1, 2], [70, 3]])
def test_caches_and_tables_without_pages(news):
    c = Case((43, len(news)), [90, 200], news, 2, 2, 64, 16, torch.float32)
    q, (table, lengths, offsets) = c.q.to(DEV), c.held()
    none = binding.Mx4Cache.empty(0, 2, 16, 64, DEV)
    assert bool(torch.isnan(binding.q8_mx4_attention(q, none, table, lengths, offsets)).all())
    assert bool(torch.isnan(binding.q8_mx4_attention(q, handle(c.c), table[:, :0], lengths, offsets)).all())
    k = torch.ones((c.rows, 2, 64), device=DEV)
    binding.q8_mx4_write(none, k, k, table, lengths, offsets)
    for x in binding.q8_mx4_read(none, table, lengths, offsets, c.rows):
        assert bool(torch.isnan(x).all())
    binding.q8_mx4_keep(none, table, lengths, offsets, torch.zeros((2, 1), dtype=torch.int32, device=DEV))
    binding.q8_mx4_copy(none, torch.zeros((2, 2), dtype=torch.int32, device=DEV))
    c.check(c.run())


@pytest.mark.parametrize("page", [64, 1024])
@pytest.mark.parametrize("columns", [1024, 2048])
def test_tables_at_the_border_of_one_launch(columns, page):
    for length in (columns, columns - 1, 1023):
        c = Case((46, columns, page, length), [length, 1], [1, 1], 1, 4, 128, page, torch.bfloat16)
        c.table = np.pad(c.table, ((0, 0), (0, columns)), constant_values=-1)[:, :columns // page]
        c.check(c.run())


def test_same_call_gives_the_same_bits():
    c = Case(36, [5000, 300, 9], [1, 4, 9], 2, 4, 128, 64, torch.float32, tree=True)
    cache = handle(c.c)
    first = c.run(cache)
    for _ in range(5):
        assert torch.equal(c.run(cache), first)


def test_empty_calls():
    c = Case(37, [20], [1], 1, 1, 64, 16, torch.float32)
    cache, none = handle(c.c), torch.zeros(0, dtype=torch.int32, device=DEV)
    assert binding.q8_mx4_attention(c.q[:0].to(DEV), cache, *c.held()).shape == (0, 1, 64)
    keepsake = torch.full(c.q.shape, 5.0, device=DEV)
    binding.q8_mx4_attention(c.q.to(DEV), cache, none.reshape(0, 4), none, ints([0]), out=keepsake)
    binding.q8_mx4_attention(c.q.to(DEV), cache, c.held()[0], c.held()[1], ints([0, 0]), out=keepsake)
    assert bool((keepsake == 5).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,dim", [([1], 128), ([8], 64), ([40], 64), ([40], 128), ([40], 256)])
def test_dominant_keys_without_values(news, dim, dtype):
    """A key that takes nearly all the weight, with values of zero: what is left
    of the weights, 2^-11 to 2^-35, makes the output."""
    for gap in (8, 16, 24):
        c = Case((51, dim, news[0]), [300], news, 1, 4, dim, 16, dtype)
        q = c.q.float()
        q[..., 0] = gap * dim ** 0.5
        c.q = q.to(dtype)
        c.qf = c.q.float().numpy()
        # channel 0: the low half of byte 0 of a key's row
        rows = c.c["k"].reshape(-1, dim // 2)
        rows[:, 0] &= 0xf0
        page, at = oc.slot_of(c.table, 16, 0, 3)
        c.c["k"][page, :, at] = 0
        c.c["k"][page, :, at, 0] = 2
        c.c["k_scale"][page, :, at] = 127
        flat = c.c["v"][page].reshape(1, -1)
        flat[:, np.unique(mx4.byte_of_channel("v", dim, at)[0])] = 0
        c.check(c.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 8, 40])
def test_one_visible_key_gives_its_value(news, dim):
    """Its weight w is within 2^-20 of 1 (the maximum is rounded, the score is not), and w V / w
    takes a rounding for each of w's parts, one for 1 / w and one for the product, each at most
    2^-24 of the value, 2^-23 for the quotient: 6 of 2^-24.  Rounded to 16 bits that is the value itself."""
    for dtype in TYPES:
        c = Case((54, dim, news), [news], [news], 1, 4, dim, 64, dtype, tree=True)
        c.trees = [[1] * news]
        got, want = c.run().cpu().double(), torch.from_numpy(c.want()[0])
        assert ((got - want).abs() <= (6 * 2.0 ** -24 if dtype == torch.float32 else 0) * want.abs()).all()


# ------------------------------------------------------------------ scores far apart

def far_keys(seed, news, dim, dtype, far, alpha=None):
    """A call whose context's first 64 keys of every 128 score far below the others: q is 1 in channel 0, where
    those keys hold -4 * 2^(far - 127) and zeros elsewhere, and the others 0."""
    c = Case((61, seed, dim, news), [300 + news], [news], 1, 4, dim, 16, dtype, alpha=alpha)
    q = c.q.float()
    q[..., 0] = 1
    c.q = q.to(dtype)
    c.qf = c.q.float().numpy()
    c.far = np.arange(300 + news) % 128 < 64
    c.far[300:] = False
    c.c["k"].reshape(-1, dim // 2)[:, 0] &= 0xf0       # channel 0: the low half of byte 0 of a key's row
    for pos in np.flatnonzero(c.far):
        page, at = oc.slot_of(c.table, 16, 0, int(pos))
        c.c["k"][page, :, at] = 0
        c.c["k"][page, :, at, 0] = 14
        c.c["k_scale"][page, :, at] = far
    return c


def want_of_near(c):
    """(out, spread, size) over the other keys alone."""
    def near(cache, name, table, b, length):
        return mx4.sequence(cache, name, table, b, length + int(c.far.sum()))[:, ~c.far]
    return oc.attention(c.qf, c.c, c.table, c.lengths - int(c.far.sum()), c.offsets, c.alpha, sequence=near)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 10, 30, 40])
def test_keys_that_score_far_below_the_others(news, dim, dtype):
    """Keys at -10^3 to -10^7 have no weight in f32 or in 64 bits (exp(-750) is none), so what is
    lost must not grow with them: the bound is that of the other keys alone."""
    for far in (139, 147, 152):
        c = far_keys(far, news, dim, dtype, far)
        ref, spread, size = want_of_near(c)
        assert np.abs(c.want()[0] - ref).max() <= 1e-12
        got = c.run().float().cpu().numpy()
        off = np.abs(got - ref) / bound(ref, spread, size, dtype)
        assert off.max() <= 1, f"far {far}: {off.max():.3f} of the bound"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 10, 30, 40])
def test_keys_that_score_further_below(news, dim, dtype):
    """The same at -10^9 and -10^37, where a step of f32 is more than what two weights may differ by."""
    for far in (160, 252):
        c = far_keys(far, news, dim, dtype, far)
        ref, spread, size = want_of_near(c)
        off = np.abs(c.run().float().cpu().numpy() - ref) / bound(ref, spread, size, dtype)
        assert off.max() <= 1, f"far {far}: {off.max():.3f} of the bound"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 10, 30, 40])
def test_scores_further_apart_than_the_largest_number(news, dim, dtype):
    """Keys at -2^127 and, after them, at 2^127 (alpha is 1): all the weight is on the latter, the same for each,
    since what their other channels add is less than half a step of such a score."""
    c = far_keys(1, news, dim, dtype, 252, alpha=1.0)
    for pos in np.flatnonzero(~c.far):
        page, at = oc.slot_of(c.table, 16, 0, int(pos))
        c.c["k"][page, :, at, ::dim // 32] = 0         # block 0
        c.c["k"][page, :, at, 0] = 6
        c.c["k_scale"][page, :, at, 0] = 252
    ref, spread, size = want_of_near(c)
    got = c.run().float().cpu().numpy()
    off = np.abs(got - ref) / bound(ref, spread, 0 * size, dtype)
    assert off.max() <= 1, f"{off.max():.3f} of the bound"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [1, 10, 30, 40])
@pytest.mark.parametrize("size", [1e6, 1e11, 1e30])
def test_all_scores_far_apart(size, news, dtype):
    """Every row's largest score is far above its next one, so its key's value is the output: the two are
    2^-13 of the terms' size apart or more, what they are rounded by is 16 * 2^-24 of it at most."""
    c = Case((63, news), [300 + news], [news], 1, 4, 128, 16, dtype, alpha=size)
    ref, got = c.want()[0], c.run().float().cpu().numpy()
    assert (np.abs(got - ref) <= bound(ref, np.abs(ref), np.zeros(ref.shape[:2]), dtype)).all()


# ------------------------------------------------------------------ large caches

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_loads_past_the_caches(dim, dtype):
    """A table and a cache that may hold more than the Infinity Cache (256 MB), which a call with a narrow table
    over few pages does not.  What the sequences do not own is NaN."""
    page, heads, columns = 64, 4, 40
    c = Case((71, dim), [2049, 300, 1], [1, 2, 1], heads, 4, dim, page, dtype)
    c.table = np.pad(c.table, ((0, 0), (0, columns)), constant_values=-1)[:, :columns]
    want = c.run()
    c.check(want)
    # 3 sequences of `wide` columns and as many pages: tokens x heads x dim x 17 / 16 bytes
    wide = 1 + (256 << 20) * 16 // (17 * 3 * page * heads * dim)
    cache = binding.Mx4Cache.empty(3 * wide, heads, page, dim, DEV)
    for n in NAMES:
        getattr(cache, n).fill_(255)
        getattr(cache, n)[:len(c.c["k"])] = dev(c.c[n])
    assert 2 * sum(getattr(cache, n).numel() for n in ("k", "k_scale")) > 256 << 20
    c.table = np.pad(c.table, ((0, 0), (0, wide - columns)), constant_values=-1)
    out = c.run(cache)
    c.check(out)
    assert torch.equal(out[-1], want[-1])       # one key; the others' items may be cut elsewhere


@pytest.mark.parametrize("dtype", TYPES)
def test_reads_past_the_caches(dtype):
    """Rows of more than 256 MB read back past the caches: the same bits as in smaller reads."""
    dim, heads, page = 128, 8, 64
    rows = (256 << 20) // (2 * heads * dim * (torch.finfo(dtype).bits // 8)) + 37
    pages = -(-rows // page)
    g = torch.Generator(device=DEV).manual_seed(9)
    cache = binding.Mx4Cache(*(torch.randint(*((0, 256) if n in "kv" else (100, 130)), (pages, heads, page, dim // 2 if n in "kv" else dim // 32),
                                             generator=g, device=DEV, dtype=torch.uint8) for n in NAMES))
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[None]
    k, v = binding.q8_mx4_read(cache, table, ints([rows]), ints([0, rows]), rows, dtype=dtype)
    half = rows // 2 + 5
    for first, n in ((0, half), (half, rows - half)):       # the newest n tokens of the first ones
        a, b = binding.q8_mx4_read(cache, table, ints([first + n]), ints([0, n]), n, dtype=dtype)
        assert torch.equal(a, k[first:first + n]) and torch.equal(b, v[first:first + n])
    few = np.array([0, 1, 63, 64, half, rows - 1])
    own = table[0].cpu().numpy()[few // page]
    c = {n: getattr(cache, n)[torch.from_numpy(own).long().to(DEV)].cpu().numpy() for n in NAMES}
    for i, t in enumerate(few):
        for name, got in (("k", k), ("v", v)):
            for h in (0, heads - 1):
                want = mx4.values(*mx4.get(c, name, i, h, int(t) % page))
                assert torch.equal(got[t, h].cpu(), torch.from_numpy(want).to(dtype))


def test_offsets_past_2_to_the_32():
    """Codes whose bytes lie past 2^32: written, read, kept, copied and attended to.  The pages that offsets
    without their 32nd or 33rd bit would reach are watched."""
    pages, heads, page, dim = 132000, 8, 64, 128      # 4.3 GB of codes a side
    size = heads * page * dim // 2
    assert (pages - 300) * size > 1 << 32
    cache = binding.Mx4Cache.empty(pages, heads, page, dim, DEV)
    for n in NAMES:
        getattr(cache, n).zero_()
    rng = np.random.default_rng(16)
    own = np.array([[pages - 1, 1, pages - 200, pages - 300]], np.int32)
    near = sorted({int(p) - b * (1 << 31) // size for p in own[0] if p > 1 for b in (1, 2)})
    copies = [near[0] + 7, near[-1] + 7, pages - 100, 77]
    assert all(0 <= p < pages and p not in own[0] for p in near) and not set(copies) & (set(near) | set(own[0].tolist()))
    k, kf = cc.rows_of(rng, (220, heads, dim), torch.bfloat16)
    v, vf = cc.rows_of(rng, (220, heads, dim), torch.bfloat16)
    q, qf = cc.rows_of(rng, (220, heads, dim), torch.bfloat16)
    held, offsets = (dev(own), ints([220]), ints([0, 220])), np.array([0, 220], np.int32)
    small = np.arange(4, dtype=np.int32)[None]
    c = {n: np.zeros((4, heads, page, dim // 2 if len(n) == 1 else dim // 32), np.uint8) for n in NAMES}

    def check(places):
        for n in NAMES:
            for i, p in enumerate(places):
                assert np.array_equal(getattr(cache, n)[int(p)].cpu().numpy(), c[n][i]), (n, p)
            assert not getattr(cache, n)[near].any(), n

    print("[mx4] write past 2^32", flush=True)
    binding.q8_mx4_write(cache, k.to(DEV), v.to(DEV), *held)
    mx4.write(c, kf, vf, small, [220], offsets)
    check(own[0])
    for got, want in zip(binding.q8_mx4_read(cache, *held, 220), mx4.read(c, small, [220], offsets)):
        assert torch.equal(got.cpu().double(), torch.from_numpy(want))
    kept = [3, 40, 64, 100, 150, 219]
    binding.q8_mx4_keep(cache, *held, ints([kept]))
    mx4.keep(c, small, [220], offsets, [kept])
    check(own[0])
    out = binding.q8_mx4_attention(q.to(DEV), cache, *held)
    ref, spread, size = mx4.attention(qf, c, small, [220], offsets, dim ** -0.5)
    assert (np.abs(out.float().cpu().numpy() - ref) <= bound(ref, spread, size, torch.bfloat16)).all()
    binding.q8_mx4_copy(cache, ints([[a, b] for a, b in zip(own[0].tolist(), copies)]))
    check(copies)
    check(own[0])
    assert torch.equal(binding.q8_mx4_attention(q.to(DEV), cache, ints([copies]), *held[1:]), out)


# ------------------------------------------------------------------ large offsets, graphs, streams

def test_offsets_past_32_bits():
    """Pages past 2^32 bytes of codes: written, read, kept, copied and attended to."""
    pages, heads, page, dim = 70000, 8, 64, 128      # 2.3 GB of codes a side
    cache = binding.Mx4Cache.empty(pages, heads, page, dim, DEV)
    cache.k_scale.fill_(127)
    cache.v_scale.fill_(127)
    rng = np.random.default_rng(6)
    own = np.array([[pages - 1, 1, pages - 2]], np.int32)
    k, kf = cc.rows_of(rng, (150, heads, dim), torch.bfloat16)
    q, qf = cc.rows_of(rng, (150, heads, dim), torch.bfloat16)
    held = (dev(own), ints([150]), ints([0, 150]))
    binding.q8_mx4_write(cache, k.to(DEV), k.to(DEV), *held)
    c = {n: np.zeros((3, heads, page, dim // 2 if len(n) == 1 else dim // 32), np.uint8) for n in NAMES}
    small, offsets = np.array([[0, 1, 2]], np.int32), np.array([0, 150], np.int32)
    mx4.write(c, kf, kf, small, [150], offsets)
    for n in NAMES:
        for i, p in enumerate(own[0]):
            keep = slice(None) if i < 2 else slice(0, 20)    # of the last page whole fours of tokens only
            assert np.array_equal(getattr(cache, n)[int(p), :, keep].cpu().numpy(), c[n][i][:, keep])
    ek, _ = mx4.read(c, small, [150], offsets)
    assert torch.equal(binding.q8_mx4_read(cache, *held, 150)[0].cpu().double(), torch.from_numpy(ek))
    out = binding.q8_mx4_attention(q.to(DEV), cache, *held)
    ref, spread, size = mx4.attention(qf, c, small, [150], offsets, dim ** -0.5)
    assert (np.abs(out.float().cpu().numpy() - ref) <= bound(ref, spread, size, torch.bfloat16)).all()
    binding.q8_mx4_copy(cache, ints([[pages - 1, 40], [1, pages - 7], [pages - 2, 7]]))
    again = binding.q8_mx4_attention(q.to(DEV), cache, ints([[40, pages - 7, 7]]), *held[1:])
    assert torch.equal(again, out)


def test_captured_and_replayed():
    """A captured step follows the lengths, pages, offsets and rows that its
    tensors hold at each replay; eager work of another shape runs between."""
    c = Case(38, [900, 900, 900], [1, 1, 1], 2, 4, 128, 64, torch.float32)
    c.lengths = np.array([700, 30, 129], np.int32)
    cache = handle(c.c)
    table, n, offsets = c.held()
    q, k, v = c.q.to(DEV), torch.randn((3, 2, 128), device=DEV), torch.randn((3, 2, 128), device=DEV)
    out = torch.empty_like(q)

    def step():
        binding.q8_mx4_write(cache, k, v, table, n, offsets)
        binding.q8_mx4_attention(q, cache, table, n, offsets, alpha=c.alpha, out=out)

    step()
    mx4.write(c.c, k.cpu().numpy(), v.cpu().numpy(), c.table, c.lengths, c.offsets)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    other = Case(39, [3000], [5], 1, 4, 128, 64, torch.float32, tree=True)
    for _ in range(4):
        n += 1
        for x in (q, k, v):
            x.normal_()
        other.check(other.run())
        out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        mx4.write(c.c, k.cpu().numpy(), v.cpu().numpy(), c.table, n.cpu().numpy(), c.offsets)
        c.lengths, c.qf = n.cpu().numpy(), q.cpu().numpy()
        c.check(replayed)
        out.fill_(0)
        step()
        assert torch.equal(out, replayed)


def test_streams_and_two_graphs_at_once():
    cases = [Case((41, i), [2000 + 300 * i, 90], [1, 2], 2, 4, 64, 16, torch.bfloat16) for i in range(3)]
    caches, helds, qs = [handle(c.c) for c in cases], [c.held() for c in cases], [c.q.to(DEV) for c in cases]
    torch.cuda.synchronize()
    streams, outs, graphs = [torch.cuda.Stream() for _ in cases], [], []
    for _ in range(4):
        outs = [binding.q8_mx4_attention(q, cache, *h, alpha=c.alpha, stream=s)
                for c, cache, h, q, s in zip(cases, caches, helds, qs, streams)]
    torch.cuda.synchronize()
    for c, out in zip(cases, outs):
        c.check(out)
    again = [torch.zeros_like(x) for x in outs]
    for c, cache, h, q, out in zip(cases, caches, helds, qs, again):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.q8_mx4_attention(q, cache, *h, alpha=c.alpha, out=out)
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, outs))
