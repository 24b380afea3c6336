"""The entry points of the 4-bit cache, the pages and the rotary positions refuse
wrong calls before they touch a device."""

import ctypes
import math
import os

import pytest
import torch

import test_cache_abi as ca
from quantized_decode_gemv_q8_amd import binding
from quantized_decode_gemv_q8_amd.build import LIB_PATH

pytestmark = pytest.mark.skipif(not os.path.exists(LIB_PATH), reason="libq8gemv.so not built")

FAKE = 0x10000
OK, BAD, LARGE = binding.Q8_OK, binding.Q8_ERR_INVALID, binding.Q8_ERR_TOO_LARGE


def calls(c, s, rows=5, k=FAKE, type_=0, stride=128, q_heads=4, q_stride=256, keep=FAKE, width=2, tree=None, words=0,
          alpha=1.0, work=FAKE, work_bytes=1 << 40):
    """Statuses of (write, read, keep, workspace, attention)."""
    L = binding.load()
    need = ctypes.c_int64(-1)
    return (L.q8_mx4_write(c, k, k, type_, rows, stride, stride, s, None),
            L.q8_mx4_read(c, k, k, type_, rows, stride, stride, s, None),
            L.q8_mx4_keep(c, rows, s, keep, width, None),
            L.q8_mx4_attention_workspace(c, type_, rows, q_heads, s, need),
            L.q8_mx4_attention(c, k, k, type_, rows, q_heads, q_stride, q_stride, s, tree, words, alpha, work,
                               work_bytes, None))


@pytest.mark.parametrize("bad", [dict(pages=-1), dict(heads=0), dict(dim=32), dict(dim=96), dict(dim=512), dict(page_size=8),
                                 dict(page_size=48), dict(page_size=2048), dict(K=None), dict(KS=None), dict(V=None),
                                 dict(VS=None), dict(K=FAKE + 8), dict(V=FAKE + 1), dict(KS=FAKE + 4), dict(VS=FAKE + 8)])
def test_bad_caches(bad):
    assert calls(ca.cache(**bad), ca.seqs()) == (BAD,) * 5


def test_null_and_bad_sequences():
    assert calls(None, ca.seqs()) == (BAD,) * 5
    assert calls(ca.cache(), None) == (BAD,) * 5
    for bad in (dict(seqs=-1), dict(max_pages=-1), dict(table_stride=2), dict(table=None), dict(lengths=None),
                dict(offsets=None), dict(table=FAKE + 2), dict(lengths=FAKE + 1), dict(offsets=FAKE + 3)):
        assert calls(ca.cache(), ca.seqs(**bad)) == (BAD,) * 5, bad


def test_sizes_past_the_limits():
    assert calls(ca.cache(pages=1 << 31), ca.seqs()) == (LARGE,) * 5
    assert calls(ca.cache(heads=65536), ca.seqs(), q_heads=65536) == (LARGE,) * 5
    assert calls(ca.cache(), ca.seqs(), rows=1 << 31) == (LARGE,) * 5
    assert calls(ca.cache(), ca.seqs(seqs=1 << 30)) == (LARGE,) * 5
    assert calls(ca.cache(), ca.seqs(max_pages=1 << 26, table_stride=1 << 26)) == (LARGE,) * 5


def test_bad_rows_keeps_and_queries():
    assert calls(ca.cache(), ca.seqs(), rows=-1) == (BAD,) * 5
    for kw in (dict(type_=3), dict(k=None), dict(k=FAKE + 2), dict(stride=127, q_stride=255)):
        st = calls(ca.cache(), ca.seqs(), **kw)
        assert (st[0], st[1], st[4]) == (BAD,) * 3, kw
    for kw in (dict(keep=None), dict(keep=FAKE + 2), dict(width=-1)):
        assert calls(ca.cache(), ca.seqs(), **kw)[2] == BAD, kw
    assert calls(ca.cache(), ca.seqs(), width=1 << 30)[2] == LARGE
    for kw in (dict(q_heads=3), dict(q_heads=0)):
        assert calls(ca.cache(), ca.seqs(), **kw)[3:] == (BAD,) * 2, kw
    for kw in (dict(words=-1), dict(tree=FAKE + 4, words=1), dict(alpha=math.inf), dict(alpha=-math.inf), dict(alpha=math.nan)):
        assert calls(ca.cache(), ca.seqs(), **kw)[4] == BAD, kw


def test_nothing_to_do_touches_nothing():
    assert calls(ca.cache(), ca.seqs(), rows=0, k=None) == (OK,) * 5
    assert calls(ca.cache(), ca.seqs(seqs=0, lengths=None, offsets=None, table=None)) == (OK,) * 5
    assert calls(ca.cache(), ca.seqs(), width=0)[2] == OK


# ------------------------------------------------------------------ copies and pages

def test_copies():
    L = binding.load()
    for f in (L.q8_cache_copy, L.q8_mx4_copy):
        assert f(None, FAKE, 3, None) == BAD
        assert f(ca.cache(dim=96), FAKE, 3, None) == BAD
        assert f(ca.cache(K=None), FAKE, 3, None) == BAD
        assert f(ca.cache(V=FAKE + 8), FAKE, 3, None) == BAD
        assert f(ca.cache(), None, 3, None) == BAD
        assert f(ca.cache(), FAKE + 2, 3, None) == BAD
        assert f(ca.cache(), FAKE, -1, None) == BAD
        assert f(ca.cache(), FAKE, 1 << 31, None) == LARGE
        assert f(ca.cache(), None, 0, None) == OK
        assert f(ca.cache(pages=0, K=None, KS=None, V=None, VS=None), None, 3, None) == OK
    assert L.q8_mx4_copy(ca.cache(KS=FAKE + 4), FAKE, 3, None) == BAD
    assert L.q8_cache_copy(ca.cache(KS=FAKE + 2), FAKE, 3, None) == BAD


def pool(**kw):
    f = dict(refs=FAKE, pages=9, page_size=16)
    f.update(kw)
    return binding._PoolStruct(*f.values())


def table(**kw):
    f = dict(table=FAKE, seqs=2, max_pages=3, table_stride=3)
    f.update(kw)
    return binding._TableStruct(*f.values())


def page_calls(p, t, a=FAKE, b=FAKE, m=FAKE, n=FAKE, work=FAKE, work_bytes=1 << 40):
    """Statuses of (fork, resize, compact)."""
    L = binding.load()
    return (L.q8_pages_fork(p, t, a, b, t, n, None),
            L.q8_pages_resize(p, t, a, b, m, n, work, work_bytes, None),
            L.q8_pages_compact(p, t, a, b, t, m, n, work, work_bytes, None))


def test_page_operations():
    for p, t in ((None, table()), (pool(), None)):
        assert page_calls(p, t) == (BAD,) * 3
    for bad in (dict(refs=None), dict(refs=FAKE + 1), dict(pages=-1), dict(page_size=8), dict(page_size=0), dict(page_size=24),
                dict(page_size=2048), dict(page_size=-16)):
        assert page_calls(pool(**bad), table()) == (BAD,) * 3, bad
    for bad in (dict(table=None), dict(table=FAKE + 2), dict(seqs=-1), dict(max_pages=-1), dict(table_stride=2)):
        assert page_calls(pool(), table(**bad)) == (BAD,) * 3, bad
    for kw in (dict(a=None), dict(b=None), dict(n=None), dict(a=FAKE + 2), dict(b=FAKE + 1), dict(n=FAKE + 3)):
        assert page_calls(pool(), table(), **kw) == (BAD,) * 3, kw
    for kw in (dict(m=None), dict(m=FAKE + 2), dict(work=None), dict(work=FAKE + 8), dict(work_bytes=0), dict(work_bytes=-1)):
        assert page_calls(pool(), table(), **kw)[1:] == (BAD,) * 2, kw
    assert page_calls(pool(pages=1 << 31), table()) == (LARGE,) * 3
    assert page_calls(pool(), table(seqs=1 << 30)) == (LARGE,) * 3
    assert page_calls(pool(), table(max_pages=1 << 26, table_stride=1 << 26)) == (LARGE,) * 3
    L = binding.load()
    assert L.q8_pages_compact(pool(), table(), FAKE, FAKE, table(seqs=3), FAKE, FAKE, FAKE, 1 << 40, None) == BAD
    assert L.q8_pages_compact(pool(), table(), FAKE, FAKE, table(max_pages=2), FAKE, FAKE, FAKE, 1 << 40, None) == BAD
    assert L.q8_pages_fork(pool(), table(), FAKE, FAKE, table(seqs=0), None, None) == OK
    assert page_calls(pool(), table(seqs=0, table=None), a=None, b=None, m=None, n=None)[:2] == (OK,) * 2


def test_workspace_sizes():
    L, n = binding.load(), ctypes.c_int64(-1)
    assert L.q8_pages_workspace(9, 2, None) == BAD
    assert L.q8_pages_workspace(-1, 2, n) == BAD and L.q8_pages_workspace(9, -1, n) == BAD
    assert L.q8_pages_workspace(1 << 31, 2, n) == LARGE and L.q8_pages_workspace(9, 1 << 30, n) == LARGE
    last = 0
    for pages, seqs in ((0, 1), (1, 1), (4097, 1), (4097, 1025), (1 << 20, 4096)):
        assert L.q8_pages_workspace(pages, seqs, n) == OK
        assert n.value > last and n.value >= 4 * pages + 8 * seqs
        last = n.value


# ------------------------------------------------------------------ rotary positions

def rope(positions=FAKE, seqs=None, n=2, type_=0, rows=5, dim=64, angles=None, x=None, **kw):
    a = dict(turns=FAKE, rot=32, interleaved=0, amplitude=1.0)
    a.update(angles or {})
    r = dict(x=FAKE, out=FAKE, heads=2, x_stride=128, out_stride=128)
    r.update(x or {})
    rows_ = (binding._RopeRowsStruct * 4)(*[tuple(r.values())] * 4)
    return binding.load().q8_rope(binding._AnglesStruct(*a.values()), rows_, n, type_, rows, dim, positions, seqs, 0, None)


def test_rope_calls():
    L = binding.load()
    assert L.q8_rope(None, None, 1, 0, 5, 64, FAKE, None, 0, None) == BAD
    for kw in (dict(n=0), dict(n=5), dict(type_=3), dict(type_=-1), dict(rows=-1), dict(dim=0), dict(dim=30), dict(positions=None),
               dict(positions=FAKE + 2), dict(seqs=ca.seqs()), dict(positions=None, seqs=ca.seqs(seqs=-1)),
               dict(positions=None, seqs=ca.seqs(lengths=None)), dict(positions=None, seqs=ca.seqs(offsets=FAKE + 1)),
               dict(angles=dict(turns=None)), dict(angles=dict(turns=FAKE + 4)), dict(angles=dict(rot=0)),
               dict(angles=dict(rot=31)), dict(angles=dict(rot=-2)), dict(angles=dict(rot=66)), dict(x=dict(x=None)),
               dict(x=dict(out=None)), dict(x=dict(x=FAKE + 2)), dict(x=dict(out=FAKE + 1)), dict(x=dict(heads=-1)),
               dict(x=dict(x_stride=127)), dict(x=dict(out_stride=127)), dict(x=dict(out_stride=130))):
        assert rope(**kw) == BAD, kw
    assert rope(dim=4098, x=dict(x_stride=1 << 14, out_stride=1 << 14)) == LARGE
    assert rope(rows=1 << 31) == LARGE
    assert rope(x=dict(heads=(1 << 20) + 1, x_stride=1 << 40, out_stride=1 << 40)) == LARGE
    assert rope(positions=None, seqs=ca.seqs(seqs=1 << 30)) == LARGE
    for kw in (dict(rows=0, positions=None), dict(x=dict(heads=0, x=None, out=None)), dict(positions=None, seqs=ca.seqs(seqs=0))):
        assert rope(**kw) == OK, kw


def test_rope_turns():
    L = binding.load()
    f = (ctypes.c_double * 6)(math.pi, 2 * math.pi, -math.pi / 2, 1.0, 0.0, 1e-9)
    out = (ctypes.c_uint64 * 6)()
    assert L.q8_rope_turns(f, 6, out) == OK
    # pi as a double is off by 2^-53 of itself
    want = [1 << 63, 0, 3 << 62, (1 << 64) / (2 * math.pi), 0, (1 << 64) * 1e-9 / (2 * math.pi)]
    for got, w in zip(out, want):
        assert min(abs(got - w), 2 ** 64 - abs(got - w)) <= 2 ** 13
    assert L.q8_rope_turns(None, 0, None) == OK
    assert L.q8_rope_turns(None, 1, out) == BAD and L.q8_rope_turns(f, -1, out) == BAD
    f[2] = math.nan
    assert L.q8_rope_turns(f, 6, out) == BAD


def test_rope_frequencies():
    F = binding.Rope.frequencies
    plain = F(64, 10000.0)
    assert plain == pytest.approx([10000 ** (-i / 32) for i in range(32)], rel=1e-14)
    assert F(64, 10000.0, "linear", 4.0) == pytest.approx([x / 4 for x in plain], rel=1e-14)
    base = F(64, 10000.0, "base", 4.0)
    assert base[0] == 1.0 and base[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)
    turns = F(64, 10000.0, "turns", 8.0, 4096)
    index = F(64, 10000.0, "index", 8.0, 4096)
    for i, x in enumerate(plain):
        r = 4096 * x / (2 * math.pi)
        w = min(max((r - 1) / 3, 0), 1)
        assert turns[i] == pytest.approx(x * w + x / 8 * (1 - w), rel=1e-13)
        if r >= 32 * 1.4:
            assert index[i] == x
        if r <= 1 / 1.4:
            assert index[i] == pytest.approx(x / 8, rel=1e-14)
        assert x / 8 * 0.999999 <= index[i] <= x
    assert F(2) == [1.0]
    for kw in (dict(rot=0), dict(rot=3), dict(rot=8, base=1.0), dict(rot=8, base=math.inf), dict(rot=2, scaling="base", factor=2.0),
               dict(rot=8, scaling="linear", factor=0.0), dict(rot=8, scaling="turns", factor=2.0), dict(rot=8, scaling="index", factor=2.0, length=-1.0),
               dict(rot=8, scaling="turns", factor=2.0, length=100.0, low=4.0, high=2.0)):
        with pytest.raises(binding.Q8Error):
            F(**kw)
    with pytest.raises(ValueError, match="scaling"):
        F(8, scaling="other")


# ------------------------------------------------------------------ without a device

_NO_DEVICE = r"""
import sys
sys.path[:0] = sys.argv[1:3]
import test_cache_abi as ca
import test_mx4_abi as t
L = t.binding.load()
print(*t.calls(ca.cache(), ca.seqs()), *t.page_calls(t.pool(), t.table()), t.rope(), L.q8_cache_copy(ca.cache(), t.FAKE, 3, None),
      L.q8_mx4_copy(ca.cache(), t.FAKE, 3, None))
"""


def test_valid_calls_without_a_device_return_an_error():
    """In a child process with every GPU hidden: an error status, no crash."""
    import subprocess
    import sys

    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible: the fake pointers would be dereferenced")
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    res = subprocess.run([sys.executable, "-c", _NO_DEVICE, os.path.dirname(here), here], capture_output=True, text=True,
                         timeout=120, env=env)
    assert res.returncode == 0, res.stderr
    statuses = [int(x) for x in res.stdout.split()]
    assert len(statuses) == 11
    assert all(s in (binding.Q8_ERR_HIP, binding.Q8_ERR_UNSUPPORTED_DEVICE) for s in statuses), statuses


# ------------------------------------------------------------------ the binding

def test_handles_check_their_tensors():
    u8 = torch.uint8
    k, ks = torch.zeros((3, 2, 16, 32), dtype=u8), torch.zeros((3, 2, 16, 2), dtype=u8)
    with pytest.raises(TypeError):
        binding.Mx4Cache(None, ks, k, ks)
    with pytest.raises(ValueError, match="dim must be"):
        binding.Mx4Cache(k[..., :16].contiguous(), ks, k, ks)
    with pytest.raises(ValueError, match="device tensor"):
        binding.Mx4Cache(k, ks, k.clone(), ks.clone())
    with pytest.raises(ValueError, match="uint8"):
        binding.Mx4Cache(k.to(torch.int8), ks, k, ks)


def handle(kind):
    c = object.__new__(kind)
    c.device, c.heads, c.dim, c.page_size, c.pages = torch.device("cuda", 0), 2, 64, 16, 3
    return c


def test_the_caches_are_not_mixed_up():
    rows, held = torch.zeros((5, 2, 64)), (torch.zeros((2, 3), dtype=torch.int32),) * 3
    for c, prefix in ((handle(binding.Q8Cache), "q8_mx4_"), (handle(binding.Mx4Cache), "q8_cache_")):
        f = {n: getattr(binding, prefix + n) for n in ("write", "read", "keep", "attention", "copy")}
        for call in (lambda: f["write"](c, rows, rows, *held), lambda: f["read"](c, *held, 5), lambda: f["keep"](c, *held, held[0]),
                     lambda: f["attention"](rows, c, *held), lambda: f["copy"](c, held[0])):
            with pytest.raises(TypeError, match="must be a"):
                call()


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    c, i32 = handle(binding.Mx4Cache), torch.int32
    rows, held = torch.zeros((5, 2, 64)), (torch.zeros((2, 3), dtype=i32),) * 3
    r = object.__new__(binding.Rope)
    r.device = torch.device("cuda", 0)
    for call in (lambda: binding.q8_mx4_write(c, rows, rows, *held, stream=Stream()),
                 lambda: binding.q8_mx4_read(c, *held, 5, stream=Stream()),
                 lambda: binding.q8_mx4_keep(c, *held, held[0], stream=Stream()),
                 lambda: binding.q8_mx4_attention(rows, c, *held, stream=Stream()),
                 lambda: binding.q8_mx4_copy(c, held[0], stream=Stream()),
                 lambda: binding.q8_rope(rows, r, positions=held[0], stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_what_is_written_stays_apart():
    a = torch.zeros(40, dtype=torch.int32)
    binding._all_apart([("x", a[:10]), ("y", a[10:20])], [("z", a[20:])])
    for bad in ([("x", a[:10]), ("y", a[9:20])], [("x", a[:10]), ("y", a[12:21])]):
        with pytest.raises(ValueError, match="overlaps"):
            binding._all_apart(bad, [("z", a[20:])])


def test_page_tables_are_checked():
    cpu, i32 = torch.device("cpu"), torch.int32
    t = binding._table("table", torch.zeros((2, 9), dtype=i32)[:, 2:5], cpu)
    assert (t.seqs, t.max_pages, t.table_stride) == (2, 3, 9)
    for bad in (torch.zeros((2, 3)), torch.zeros(3, dtype=i32), torch.zeros((3, 4), dtype=i32).t(),
                torch.zeros(4, dtype=i32).as_strided((2, 3), (1, 1))):
        with pytest.raises(ValueError):
            binding._table("table", bad, cpu)
    with pytest.raises(TypeError):
        binding._table("table", None, cpu)


def test_rope_rows_are_checked():
    cpu, f32 = torch.device("cpu"), torch.float32
    wide = torch.zeros((5, 300))[:, 3:131].unflatten(1, (2, 64))
    assert binding._rope_rows("x", wide, 5, 64, f32, cpu) == 300
    assert binding._rope_rows("x", torch.zeros((5, 2, 64)), 5, 64, None, cpu) == 128
    for bad in (wide.double(), wide.half(), torch.zeros((4, 2, 64)), torch.zeros((5, 2, 32)), torch.zeros((5, 64, 2)).transpose(1, 2),
                torch.zeros(64 * 8).as_strided((5, 2, 64), (64, 64, 1))):
        with pytest.raises(ValueError):
            binding._rope_rows("x", bad, 5, 64, f32, cpu)
    with pytest.raises(TypeError):
        binding._rope_rows("x", 1, 5, 64, f32, cpu)


@pytest.mark.parametrize("given", [False, True])
def test_rope_positions_are_checked_before_they_are_used(given):
    """Whether or not there is an output to keep apart from them."""
    x, one = torch.zeros((4, 2, 64)), torch.zeros(4, dtype=torch.int32)
    r = binding.Rope([1.0] * 32, device="cpu")
    kw = dict(out=torch.zeros((4, 2, 64))) if given else {}
    for bad in (dict(positions=[0, 1, 2, 3]), dict(positions=3), dict(lengths=[4], offsets=[0, 4]), dict(lengths=one, offsets=[0, 4]),
                dict()):
        with pytest.raises(TypeError):
            binding.q8_rope(x, r, **bad, **kw)
    for bad in (dict(positions=one, lengths=one), dict(positions=one.long()), dict(positions=one), dict(lengths=one, offsets=one),
                dict(lengths=one[None], offsets=one)):
        with pytest.raises(ValueError):
            binding.q8_rope(x, r, **bad, **kw)
