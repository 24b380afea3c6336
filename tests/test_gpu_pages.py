"""Forking, resizing, compacting and copying pages on the GPU, against the plain
Python reference, number for number."""

import numpy as np
import pytest
import torch

import cache_cases as cc
import mx4_cases as mc
from oracle import mx4, pages
from quantized_decode_gemv_q8_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pool(seed, n_pages, lengths, page_size, columns, share=0.0):
    """refs and table of sequences whose pages are random ones, some shared with the sequence before."""
    rng = np.random.default_rng(seed)
    order, at = rng.permutation(n_pages).tolist(), 0
    refs, table = [0] * n_pages, []
    for b, n in enumerate(lengths):
        row = []
        for c in range(pages.pages_of(max(n, 0), page_size)):
            if b and rng.random() < share and c < len(table[-1]) and table[-1][c] >= 0:
                row.append(table[-1][c])
            else:
                row.append(order[at])
                at += 1
            refs[row[-1]] += 1
        table.append(row + [-1] * (columns - len(row)))
    return rng, refs, table


def check_resize(refs, table, before, after, page_size, apart=0):
    """Runs a resize and compares everything; returns the new (refs, table, moves, missing)."""
    want = pages.resize(refs, table, before, after, page_size)
    wide = torch.full((len(table), len(table[0]) + apart), 77, dtype=torch.int32, device=DEV)
    t = wide[:, :len(table[0])]
    t.copy_(ints(table))
    r = ints(refs)
    moves, missing = binding.q8_pages_resize(r, t, ints(before), ints(after), page_size)
    for got, w, name in ((r, want[0], "refs"), (t, want[1], "table"), (moves, want[2], "moves"), (missing, want[3], "missing")):
        assert got.tolist() == w, name
    assert bool((wide[:, len(table[0]):] == 77).all())
    return want


SIZES = [(9, 3, 4, 16), (70, 30, 9, 32), (5000, 1100, 12, 16), (40000, 300, 40, 64), (40000, 2500, 20, 16)]


@pytest.mark.parametrize("which", range(len(SIZES)))
@pytest.mark.parametrize("share", [0.0, 0.5])
def test_resize(which, share):
    """Sequences that grow, shrink, stay, come and leave at once; small pools and large ones."""
    n_pages, seqs, columns, page = SIZES[which]
    rng = np.random.default_rng((1, which))
    most = min(columns * page, int(1.6 * n_pages * page / seqs))
    before = [int(x) for x in rng.integers(0, most + 1, seqs)]
    while sum(pages.pages_of(n, page) for n in before) > n_pages:
        before = [n // 2 for n in before]
    after = [int(min(columns * page, max(0, n + x))) for n, x in zip(before, rng.integers(-2 * page, 2 * page, seqs))]
    for b in rng.integers(0, seqs, seqs // 3):
        after[b] = int(rng.choice([0, before[b], min(before[b] + 1, columns * page)]))
    _, refs, table = pool((2, which), n_pages, before, page, columns, share)
    print(f"[pages] resize {which} share {share}", flush=True)
    refs, table, _, missing = check_resize(refs, table, before, after, page, apart=which % 2)
    held = [a if m == 0 else b for a, b, m in zip(after, before, missing)]
    check_resize(refs, table, held, [0] * seqs, page)           # everyone leaves


def test_growing_a_step_at_a_time():
    """Token by token over page borders, until the pool is empty; then one leaves and the others go on."""
    page, columns = 16, 4
    lengths, refs, table = [15, 16, 17, 0], [0] * 9, [[-1] * columns for _ in range(4)]
    refs, table, _, _ = check_resize(refs, table, [0] * 4, lengths, page)
    seen = False
    for step in range(40):
        after = [n + (1 + b if n + 1 + b <= columns * page else 0) for b, n in enumerate(lengths)]
        refs, table, _, missing = check_resize(refs, table, lengths, after, page)
        lengths = [a if m == 0 else n for a, n, m in zip(after, lengths, missing)]
        if any(missing) and not seen:
            seen = True
            refs, table, _, _ = check_resize(refs, table, lengths, [0] + lengths[1:], page)
            lengths[0] = 0
    assert seen


def test_shared_last_pages_are_replaced():
    """Two, three and all owners of a partly filled page grow at once; a full one is not replaced;
    one whose other owner leaves in the same call keeps it."""
    page = 16
    for growing in ([0, 1], [0, 1, 2], [2]):
        table = [[3, 5, -1], [3, 5, -1], [3, 5, -1]]
        refs = [0] * 10
        refs[3] = refs[5] = 3
        before = [20, 20, 20]
        check_resize(refs, table, before, [n + 1 if b in growing else n for b, n in enumerate(before)], page)
        check_resize(refs, table, [32] * 3, [33 if b in growing else 32 for b in range(3)], page)
    table, refs = [[3, -1], [3, -1]], [0] * 6
    refs[3] = 2
    _, _, moves, _ = check_resize(refs, table, [5, 5], [0, 6], page)
    assert moves == [[-1, -1], [-1, -1]]


def test_wrong_descriptions_are_left_alone():
    page = 16
    table = [[0, 1, -1], [2, 99, -1], [-1, 3, 4], [5, 6, 7]]
    refs = [1] * 8 + [0] * 4
    for before, after in (([-1, 20, 20, 20], [5, 40, 40, 40]), ([20, 20, 20, 49], [20, 49, -3, 20]),
                          ([20, 40, 5, 2 ** 31 - 1], [0, 0, 0, 0]), ([20, 20, 5, 48], [21, 21, 6, -2 ** 31])):
        check_resize(refs, table, before, after, page)


@pytest.mark.parametrize("n_pages,takes,columns", [(9000, [4095], 5000), (9000, [4096, 3], 5000), (9000, [1, 5000, 2], 5001),
                                                   (9000, [3000, 3000], 9000), (131072, [5, 70], 90), (131073, [5, 70], 90)])
def test_many_pages_at_once(n_pages, takes, columns):
    """More pages than one workgroup lists on the chip, and the borders of what one workgroup does."""
    page = 16
    _, refs, table = pool((9, n_pages, len(takes)), n_pages, [0] * len(takes), page, columns)
    rng = np.random.default_rng((10, n_pages))
    for p in rng.choice(n_pages, n_pages // 3, replace=False):
        refs[p] = 1                                     # owned by rows of another table
    after = [n * page - 3 for n in takes]
    print(f"[pages] {takes} of {n_pages}", flush=True)
    refs, table, _, missing = check_resize(refs, table, [0] * len(takes), after, page)
    assert missing == [0] * len(takes)
    check_resize(refs, table, after, [0, 4 * page] + [0] * (len(takes) - 2) if len(takes) > 1 else [20], page)


@pytest.mark.parametrize("n_pages", [81920, 81921])
def test_free_pages_that_come_last(n_pages):
    """On both sides of what one workgroup looks through; all pages but the last 80 have owners."""
    page, lengths = 16, [24, 16, 24, 0, 160]
    _, refs, table = pool((15, n_pages), n_pages - 80, lengths, page, 60, share=0.5)
    refs = [max(x, 1) for x in refs] + [0] * 80
    refs, table, _, missing = check_resize(refs, table, lengths, [40, 100, 25, 900, 0], page)
    assert missing == [0, 0, 0, 0, 0]
    _, _, _, missing = check_resize(refs, table, [40, 100, 25, 900, 0], [60, 120, 0, 940, 500], page)
    assert missing[-1] > 0


def test_more_tiles_than_workgroups():
    """Pools and batches of which a workgroup takes several tiles, and more children than a grid has waves."""
    n_pages, seqs, columns, page = 2_200_000, 530_000, 4, 16
    rng = np.random.default_rng(12)
    before = rng.integers(0, 3 * page, seqs)
    after = np.maximum(before + rng.integers(-20, 21, seqs), 0).tolist()
    before = before.tolist()
    _, refs, table = pool(13, n_pages, before, page, columns)
    print("[pages] large resize", flush=True)
    refs, table, _, missing = check_resize(refs, table, before, after, page)
    assert missing == [-1 if n > columns * page else 0 for n in after]
    print("[pages] large compact", flush=True)
    want = pages.compact(refs, table, after, page)
    got = binding.q8_pages_compact(ints(refs), ints(table), ints(after), page)
    for g, w, name in zip(got, (want[0], want[1], want[2], [want[3]]), ("refs", "table", "moves", "used")):
        assert torch.equal(g.cpu(), torch.tensor(w, dtype=torch.int32)), name
    children = (1 << 22) + 9
    parent = torch.arange(children, dtype=torch.int32, device=DEV) % 3
    count = ints([0] * 5)
    print("[pages] many children", flush=True)
    t, n = binding.q8_pages_fork(count, ints([[4], [-1], [2]]), ints([3, 0, 16]), parent, page)
    assert torch.equal(t[:, 0], ints([4, -1, 2])[parent.long()]) and torch.equal(n, ints([3, 0, 16])[parent.long()])
    assert count.tolist() == [0, 0, int((parent == 2).sum()), 0, int((parent == 0).sum())]


def test_table_rows_past_32_bits():
    """Rows of a table whose bytes lie past 2^33."""
    page, wide = 16, (1 << 30) + 16
    room = torch.empty(2 * wide + 8, dtype=torch.int32, device=DEV)
    far = room.as_strided((3, 4), (wide, 1))
    table = [[5, 1, -1, -1], [3, -1, -1, -1], [0, 2, -1, -1]]
    refs = [1, 1, 1, 1, 0, 1, 0, 0, 0, 0]
    before, after = [20, 16, 32], [50, 0, 40]
    far.copy_(ints(table))
    r = ints(refs)
    print("[pages] rows far apart", flush=True)
    moves, missing = binding.q8_pages_resize(r, far, ints(before), ints(after), page)
    want = pages.resize(refs, table, before, after, page)
    for got, w in zip((r, far, moves, missing), want):
        assert got.tolist() == w
    got = binding.q8_pages_compact(r, far, ints(after), page)
    assert got[1].tolist() == pages.compact(want[0], want[1], after, page)[1]
    children = pages.fork(want[0], want[1], after, [2, 0, 2], page, 4)
    t, n = binding.q8_pages_fork(r, far, ints(after), ints([2, 0, 2]), page)
    assert t.tolist() == children[1] and n.tolist() == children[2] and r.tolist() == children[0]


def test_pools_and_tables_of_nothing():
    none = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    refs = ints([1, 0])
    moves, missing = binding.q8_pages_resize(refs, none, ints([]), ints([]), 16)
    assert moves.shape == (0, 2) and missing.shape == (0,)
    check_resize([], [[-1, -1]], [0], [17], 16)                                  # a pool of no pages
    moves, missing = binding.q8_pages_resize(refs, none.reshape(3, 0), ints([0, 0, 1]), ints([0, 1, 0]), 16)
    assert missing.tolist() == [0, -1, -1]
    t, n = binding.q8_pages_fork(refs, none, ints([]), ints([0, -1]), 16)
    assert n.tolist() == [0, 0] and t.tolist() == [[-1] * 3] * 2
    for k in (0, 1):
        r, t, m, u = binding.q8_pages_compact(ints([3] * k), none, ints([]), 16)
        assert r.tolist() == [3] * k and m.shape == (0, 2) and u.tolist() == [k]


@pytest.mark.parametrize("seqs,children,columns", [(1, 1, 3), (5, 40, 9), (300, 1000, 70)])
def test_fork(seqs, children, columns):
    rng = np.random.default_rng((3, seqs))
    page = 16
    lengths = [int(x) for x in rng.integers(0, columns * page + 1, seqs)]
    n_pages = sum(pages.pages_of(n, page) for n in lengths) + 5
    _, refs, table = pool((4, seqs), n_pages, lengths, page, columns, 0.3)
    lengths += [-4, columns * page + 1, 2 ** 31 - 1]
    table += [[0] * columns] * 3
    if lengths[0] > page:
        table[0][1] = -1                    # entries that are no page
        table[0][0] = n_pages
    parent = [int(x) for x in rng.integers(0, seqs + 3, children)] + [-1, seqs + 3, -2 ** 31, 2 ** 31 - 1]
    for out_columns in (columns, columns + 4, max(1, columns - 2)):
        want = pages.fork(refs, table, lengths, parent, page, out_columns)
        r, t = ints(refs), torch.full((len(parent), out_columns), 9, dtype=torch.int32, device=DEV)
        got, n = binding.q8_pages_fork(r, ints(table), ints(lengths), ints(parent), page, table_out=t)
        assert got is t and got.tolist() == want[1] and n.tolist() == want[2] and r.tolist() == want[0]


@pytest.mark.parametrize("n_pages,seqs,columns", [(1, 1, 1), (7, 2, 2), (300, 20, 9), (4096, 100, 30), (40001, 700, 33),
                                                   (4096, 64, 64), (4096, 64, 65), (4097, 10, 300)])
@pytest.mark.parametrize("fill", [0.1, 0.5, 0.97, 1.0])
def test_compact(n_pages, seqs, columns, fill):
    rng = np.random.default_rng((5, n_pages, int(100 * fill)))
    page = 16
    lengths = [int(x) for x in rng.integers(0, columns * page + 1, seqs)]
    while sum(pages.pages_of(n, page) for n in lengths) > fill * n_pages:
        lengths = [n // 2 for n in lengths]
    _, refs, table = pool((6, n_pages), n_pages, lengths, page, columns, 0.2)
    spare = [p for p in range(n_pages) if refs[p] == 0]
    for p in rng.permutation(spare)[:max(0, int(fill * n_pages) - (n_pages - len(spare)))]:
        refs[p] = int(rng.integers(1, 4))               # owned by rows of another table
    for p in [p for p in range(n_pages) if refs[p] == 0][:3]:
        refs[p] = -1
    lengths[0] = -3 if seqs > 4 else lengths[0]
    want = pages.compact(refs, table, lengths, page)
    r, t = ints(refs), ints(table)
    got = binding.q8_pages_compact(r, t, ints(lengths), page)
    for g, w, name in zip(got, (want[0], want[1], want[2], [want[3]]), ("refs", "table", "moves", "used")):
        assert g.tolist() == w, name
    assert r.tolist() == refs and t.tolist() == table


def caches(heads, page, dim, n_pages):
    g = torch.Generator(device=DEV)
    g.manual_seed(8)

    def some(shape, dtype):
        x = torch.randint(0, 256, (*shape, torch.empty((), dtype=dtype).element_size()), generator=g, device=DEV, dtype=torch.uint8)
        return x.view(dtype).squeeze(-1)
    shape = (n_pages, heads, page)
    return (binding.Q8Cache(*(some((*shape, n), t) for n, t in ((dim, torch.int8), (dim // 32, torch.float32)) * 2)),
            binding.Mx4Cache(*(some((*shape, n), torch.uint8) for n in (dim // 2, dim // 32) * 2)))


@pytest.mark.parametrize("heads,page,dim", [(1, 16, 64), (3, 16, 128), (8, 64, 128), (2, 1024, 256), (5, 32, 64)])
def test_copy(heads, page, dim):
    """Every byte of the pages that are moved, and of those that are not."""
    n = 40
    moves = [[3, 7], [-1, -1], [0, 39], [39 + 1, 5], [5, 40], [6, 6], [-2 ** 31, 4], [4, 2 ** 31 - 1], [38, 1], [3, 2], [-1, 8]]
    for cache in caches(heads, page, dim, n):
        want = {x: getattr(cache, x).clone() for x in ("k", "k_scale", "v", "v_scale")}
        for x in want.values():
            for a, b in ((3, 7), (0, 39), (38, 1), (3, 2)):
                x[b] = x[a]
        (binding.q8_mx4_copy if isinstance(cache, binding.Mx4Cache) else binding.q8_cache_copy)(cache, ints(moves))
        for name, x in want.items():
            assert torch.equal(getattr(cache, name).view(torch.uint8), x.view(torch.uint8)), name
    for cache, copy in zip(caches(heads, page, dim, 3), (binding.q8_cache_copy, binding.q8_mx4_copy)):
        copy(cache, ints([]).reshape(0, 2))


def test_copy_of_scales_at_any_word():
    """The Q8_0 cache's scales need only their own alignment."""
    shape = (6, 2, 16, 128)
    k = torch.randint(-127, 128, shape, dtype=torch.int8, device=DEV)
    room = torch.rand(2 * 6 * 2 * 16 * 4 + 3, device=DEV)
    n = 6 * 2 * 16 * 4
    ks, vs = room[1:1 + n].view(6, 2, 16, 4), room[2 + n:2 + 2 * n].view(6, 2, 16, 4)
    cache = binding.Q8Cache(k, ks, k.clone(), vs)
    want = [x.clone() for x in (ks, vs)]
    binding.q8_cache_copy(cache, ints([[2, 5], [0, 1]]))
    for x, w in zip((ks, vs), want):
        w[5], w[1] = w[2], w[0]
        assert torch.equal(x, w)


def test_captured_and_replayed():
    """A captured decode step grows its sequences; each replay is as the reference's step."""
    page, columns, n_pages, seqs = 16, 8, 60, 6
    lengths = [5, 16, 31, 40, 0, 64]
    _, refs, table = pool(9, n_pages, lengths, page, columns)
    r, t, before = ints(refs), ints(table), ints(lengths)
    after = before + 3
    moves, missing = torch.empty((seqs, 2), dtype=torch.int32, device=DEV), torch.empty(seqs, dtype=torch.int32, device=DEV)
    outs = [torch.empty_like(r), torch.empty_like(t), torch.empty((n_pages // 2, 2), dtype=torch.int32, device=DEV), ints([0])]
    child, child_len, parent = torch.empty_like(t), torch.empty_like(before), ints([5, 4, 3, 2, 1, 0])
    none = torch.zeros_like(before)

    def step():
        binding.q8_pages_resize(r, t, before, after, page, moves=moves, missing=missing)
        before.copy_(after)
        after.add_(3)
        binding.q8_pages_fork(r, t, before, parent, page, table_out=child, lengths_out=child_len)
        binding.q8_pages_compact(r, t, before, page, *outs)
        binding.q8_pages_resize(r, child, child_len, none, page)

    def follow():
        nonlocal refs, table, lengths
        refs, table, m, lost = pages.resize(refs, table, lengths, [n + 3 for n in lengths], page)
        lengths = [n + 3 for n in lengths]
        forked = pages.fork(refs, table, lengths, parent.tolist(), page, columns)
        packed = pages.compact(forked[0], table, lengths, page)
        assert moves.tolist() == m and missing.tolist() == lost and child_len.tolist() == forked[2]
        for got, want in zip(outs, (packed[0], packed[1], packed[2], [packed[3]])):
            assert got.tolist() == want
        assert r.tolist() == refs and t.tolist() == table and child.tolist() == [[-1] * columns] * seqs

    step()
    follow()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        binding.q8_pages_compact(ints([0, 1, 0, 2]), ints([[3, 1]]), ints([20]), 16)      # eager work between
        g.replay()
        torch.cuda.synchronize()
        follow()


def test_two_pools_on_two_streams():
    page, columns = 16, 6
    made = [pool((10, i), 5000, [50 + i] * 200, page, columns) for i in range(2)]
    state = [(ints(refs), ints(table), ints([50 + i] * 200), ints([70 + i] * 200)) for i, (_, refs, table) in enumerate(made)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [binding.q8_pages_resize(r, t, a, b, page, stream=s) for (r, t, a, b), s in zip(state, streams)]
    torch.cuda.synchronize()
    for i, (_, refs, table) in enumerate(made):
        want = pages.resize(refs, table, [50 + i] * 200, [70 + i] * 200, page)
        for g, w in zip((state[i][0], state[i][1], *got[i]), want):
            assert g.tolist() == w


@pytest.mark.parametrize("dtype", mc.TYPES)
def test_a_search_over_a_cache(dtype):
    """As a serving loop runs it: prompts rotated and written, forked into beams that share
    them, each beam grown, written to and attended with, beams dropped, the pool
    compacted, and the next step; against the reference's cache and attention."""
    heads, group, dim, page, columns, n_pages = 2, 4, 64, 16, 6, 64
    rng = np.random.default_rng(12)
    cache = binding.Mx4Cache.empty(n_pages, heads, page, dim, DEV)
    for x in (cache.k, cache.v):
        x.zero_()
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(127)
    c = {n: getattr(cache, n).cpu().numpy() for n in ("k", "k_scale", "v", "v_scale")}
    refs, table, lengths = [0] * n_pages, [[-1] * columns for _ in range(2)], [0, 0]
    r, t, n = ints(refs), ints(table), ints(lengths)
    rope = binding.Rope.scaled(dim, 10000.0, interleaved=True, device=DEV)

    def step(news):
        nonlocal refs, table, lengths, n
        after = [a + b for a, b in zip(lengths, news)]
        moves, missing = binding.q8_pages_resize(r, t, n, ints(after), page)
        binding.q8_mx4_copy(cache, moves)
        refs, table, m, lost = pages.resize(refs, table, lengths, after, page)
        assert moves.tolist() == m and missing.tolist() == lost == [0] * len(news)
        for a, b in m:
            for x in c.values():
                if a >= 0:
                    x[b] = x[a]
        lengths, n = after, ints(after)
        offsets = cc.offsets_of(news)
        rows = int(offsets[-1])
        held = (t, n, torch.from_numpy(offsets).to(DEV))
        k, q = (torch.randn((rows, h, dim), device=DEV).to(dtype) for h in (heads, heads * group))
        v = torch.randn((rows, heads, dim), device=DEV).to(dtype)
        q, k = binding.q8_rope((q, k), rope, lengths=n, offsets=held[2])
        binding.q8_mx4_write(cache, k, v, *held)
        mx4.write(c, k.float().cpu().numpy(), v.float().cpu().numpy(), np.array(table), lengths, offsets)
        for name, x in c.items():
            assert np.array_equal(getattr(cache, name).cpu().numpy(), x), name
        out = binding.q8_mx4_attention(q, cache, *held)
        ref, spread, size = mx4.attention(q.float().cpu().numpy(), c, np.array(table), lengths, offsets, dim ** -0.5)
        far = np.abs(out.float().cpu().numpy() - ref) / mc.bound(ref, spread, size, dtype)
        assert far.max() <= 1

    def fork(parent):
        nonlocal refs, table, lengths, r, t, n
        old = t, n
        t, n = binding.q8_pages_fork(r, t, n, ints(parent), page)
        gone = table, lengths
        refs, table, lengths = pages.fork(refs, table, lengths, parent, page, columns)
        binding.q8_pages_resize(r, *old, torch.zeros_like(old[1]), page)        # the parents leave
        refs = pages.resize(refs, *gone, [0] * len(gone[1]), page)[0]
        assert r.tolist() == refs and t.tolist() == table and n.tolist() == lengths

    step([37, 20])
    fork([0, 0, 1, 0, 1])
    step([1, 1, 1, 1, 1])
    step([3, 2, 1, 14, 9])
    fork([3, 3, 0])
    step([1, 1, 2])
    r, t, moves, used = binding.q8_pages_compact(r, t, n, page)
    refs, table, m, u = pages.compact(refs, table, lengths, page)
    assert r.tolist() == refs and t.tolist() == table and moves.tolist() == m and used.item() == u
    binding.q8_mx4_copy(cache, moves)
    for a, b in m:
        if a >= 0:
            for x in c.values():
                x[b] = x[a]
    assert any(a >= 0 for a, _ in m)
    step([1, 1, 1])


@pytest.mark.parametrize("dtype", mc.TYPES)
def test_a_captured_step_that_runs_out_of_pages(dtype):
    """Sequences that get no page get a length of -1 for the step, on the device: nothing of theirs is written,
    least of all into the last page that they share with others, and their rows are NaN."""
    heads, group, dim, page, columns, seqs, n_pages = 2, 2, 64, 16, 4, 4, 4
    cache = binding.Mx4Cache.empty(n_pages, heads, page, dim, DEV)
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        x.fill_(120)
    c = {n: getattr(cache, n).cpu().numpy() for n in ("k", "k_scale", "v", "v_scale")}
    # all share 24 tokens in pages 2 and 0; pages 1 and 3 are free
    refs, table, lengths, news = [4, 0, 4, 0], [[2, 0, -1, -1] for _ in range(seqs)], [24] * seqs, [1] * seqs
    r, t, before, new, offsets = ints(refs), ints(table), ints(lengths), ints(news), ints(list(range(seqs + 1)))
    q, k, v = (torch.zeros((seqs, h, dim), dtype=dtype, device=DEV) for h in (heads * group, heads, heads))
    rope = binding.Rope.scaled(dim, device=DEV)
    now = {}

    def step():
        after = before + new
        moves, missing = binding.q8_pages_resize(r, t, before, after, page)
        binding.q8_mx4_copy(cache, moves)
        now["held"] = torch.where(missing == 0, after, -1)
        now["q"], now["k"] = binding.q8_rope((q, k), rope, lengths=now["held"], offsets=offsets)
        binding.q8_mx4_write(cache, now["k"], v, t, now["held"], offsets)
        now["out"] = binding.q8_mx4_attention(now["q"], cache, t, now["held"], offsets)
        before.copy_(torch.where(missing == 0, after, before))

    def fresh():
        for x in (q, k, v):
            x.normal_()

    def follow():
        nonlocal refs, table, lengths
        after = [a + b for a, b in zip(lengths, news)]
        refs, table, moves, missing = pages.resize(refs, table, lengths, after, page)
        for a, b in moves:
            if a >= 0:
                for x in c.values():
                    x[b] = x[a]
        served = [b for b in range(seqs) if missing[b] == 0 and news[b]]
        assert now["held"].tolist() == [a if m == 0 else -1 for a, m in zip(after, missing)]
        lengths = [a if m == 0 else b for a, b, m in zip(after, lengths, missing)]
        rows, only = np.array(served), np.arange(len(served) + 1)
        host = {n: now[n].float().cpu().numpy() for n in ("q", "k", "out")}
        own = np.array(table)[rows], [lengths[b] for b in served], only
        mx4.write(c, host["k"][rows], v.float().cpu().numpy()[rows], *own)
        for name, x in c.items():
            assert np.array_equal(getattr(cache, name).cpu().numpy(), x), name
        ref, spread, size = mx4.attention(host["q"][rows], c, *own, dim ** -0.5)
        assert (np.abs(host["out"][rows] - ref) <= mc.bound(ref, spread, size, dtype)).all()
        assert np.isnan(host["out"][[b for b in range(seqs) if b not in served]]).all()
        assert r.tolist() == refs and t.tolist() == table and before.tolist() == lengths
        return served

    def leave(b):
        nonlocal refs, table, lengths
        after = [0 if i == b else n for i, n in enumerate(lengths)]
        binding.q8_pages_resize(r, t, before, ints(after), page)
        refs, table, _, _ = pages.resize(refs, table, lengths, after, page)
        lengths, news[b] = after, 0
        before.copy_(ints(after))
        new.copy_(ints(news))

    fresh()
    step()
    assert follow() == [0, 1]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for gone, want in ((None, [0, 1]), (None, [0, 1]), (0, [1, 2]), (None, [1, 2, 3]), (1, [2, 3])):
        if gone is not None:
            leave(gone)
        fresh()
        g.replay()
        torch.cuda.synchronize()
        assert follow() == want
