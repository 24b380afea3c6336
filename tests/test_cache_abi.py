"""The cache's entry points refuse wrong calls before they touch a device."""

import ctypes
import os

import pytest
import torch

from quantized_decode_gemv_q8_amd import binding
from quantized_decode_gemv_q8_amd.build import LIB_PATH

pytestmark = pytest.mark.skipif(not os.path.exists(LIB_PATH), reason="libq8gemv.so not built")

FAKE = 0x10000


def cache(**kw):
    f = dict(K=FAKE, KS=FAKE, V=FAKE, VS=FAKE, pages=4, heads=2, page_size=16, dim=64)
    f.update(kw)
    return binding._CacheStruct(*f.values())


def seqs(**kw):
    f = dict(table=FAKE, lengths=FAKE, offsets=FAKE, seqs=2, max_pages=3, table_stride=3)
    f.update(kw)
    return binding._SeqsStruct(*f.values())


def calls(c, s, rows=5, k=FAKE, type_=0, stride=128, q_heads=4, q_stride=256, keep=FAKE, width=2, tree=None, words=0,
          work=FAKE, work_bytes=1 << 40):
    """Statuses of (write, read, keep, workspace, attention)."""
    L = binding.load()
    need = ctypes.c_int64(-1)
    return (L.q8_cache_write(c, k, k, type_, rows, stride, stride, s, None),
            L.q8_cache_read(c, k, k, type_, rows, stride, stride, s, None),
            L.q8_cache_keep(c, rows, s, keep, width, None),
            L.q8_cache_attention_workspace(c, type_, rows, q_heads, s, need),
            L.q8_cache_attention(c, k, k, type_, rows, q_heads, q_stride, q_stride, s, tree, words, 1.0, work,
                                 work_bytes, None))


INVALID = (binding.Q8_ERR_INVALID,) * 5
LARGE = (binding.Q8_ERR_TOO_LARGE,) * 5


def test_null_descriptors():
    assert calls(None, seqs()) == INVALID
    assert calls(cache(), None) == INVALID


@pytest.mark.parametrize("bad", [dict(pages=-1), dict(heads=0), dict(heads=-2), dict(dim=32), dict(dim=96), dict(dim=0),
                                 dict(dim=512), dict(page_size=0), dict(page_size=8), dict(page_size=48),
                                 dict(page_size=2048), dict(page_size=-16), dict(K=None), dict(KS=None), dict(V=None),
                                 dict(VS=None), dict(K=FAKE + 8), dict(V=FAKE + 1), dict(KS=FAKE + 2), dict(VS=FAKE + 1)])
def test_bad_caches(bad):
    assert calls(cache(**bad), seqs()) == INVALID


@pytest.mark.parametrize("bad", [dict(seqs=-1), dict(max_pages=-1), dict(table_stride=2), dict(table=None),
                                 dict(lengths=None), dict(offsets=None), dict(table=FAKE + 2), dict(lengths=FAKE + 1),
                                 dict(offsets=FAKE + 3)])
def test_bad_sequences(bad):
    assert calls(cache(), seqs(**bad)) == INVALID


def test_sizes_past_the_limits():
    assert calls(cache(pages=1 << 31), seqs()) == LARGE
    assert calls(cache(heads=65536), seqs(), q_heads=65536) == LARGE
    assert calls(cache(), seqs(), rows=1 << 31) == LARGE
    assert calls(cache(), seqs(seqs=1 << 30)) == LARGE
    assert calls(cache(), seqs(max_pages=1 << 26, table_stride=1 << 26)) == LARGE


def test_bad_rows():
    assert calls(cache(), seqs(), rows=-1) == INVALID
    for kw in (dict(type_=3), dict(type_=-1), dict(k=None), dict(k=FAKE + 2)):
        st = calls(cache(), seqs(), **kw)
        assert (st[0], st[1], st[4]) == INVALID[:3], kw
    assert calls(cache(), seqs(), k=FAKE + 1, type_=1)[0] == binding.Q8_ERR_INVALID
    st = calls(cache(), seqs(), stride=127, q_stride=255)     # rows would overlap
    assert (st[0], st[1], st[4]) == INVALID[:3]


def test_bad_keep():
    assert calls(cache(), seqs(), keep=None)[2] == binding.Q8_ERR_INVALID
    assert calls(cache(), seqs(), keep=FAKE + 2)[2] == binding.Q8_ERR_INVALID
    assert calls(cache(), seqs(), width=-1)[2] == binding.Q8_ERR_INVALID
    assert calls(cache(), seqs(), width=1 << 30)[2] == binding.Q8_ERR_TOO_LARGE


def test_bad_attention():
    for kw in (dict(q_heads=3), dict(q_heads=0), dict(q_heads=-2)):
        assert calls(cache(), seqs(), **kw)[3:] == INVALID[:2], kw
    assert calls(cache(), seqs(), words=-1)[4] == binding.Q8_ERR_INVALID
    assert calls(cache(), seqs(), tree=FAKE + 4, words=1)[4] == binding.Q8_ERR_INVALID
    assert binding.load().q8_cache_attention_workspace(cache(), 0, 5, 4, seqs(), None) == binding.Q8_ERR_INVALID


def test_attention_past_the_work_list():
    """More units of work than the list can number; the same sizes alone are allowed."""
    for kw in (dict(seqs=1 << 29, max_pages=1, table_stride=1), dict(seqs=1 << 12, max_pages=1 << 25, table_stride=1 << 25)):
        st = calls(cache(heads=256), seqs(**kw), rows=(1 << 31) - 1, q_heads=256, q_stride=1 << 14)
        assert st[3:] == LARGE[:2], kw
    st = calls(cache(), seqs(), q_heads=1 << 25, q_stride=1 << 31)
    assert st[3:] == LARGE[:2]


def test_nothing_to_do_touches_nothing():
    ok = (binding.Q8_OK,) * 5
    assert calls(cache(), seqs(), rows=0, k=None) == ok
    assert calls(cache(), seqs(seqs=0, lengths=None, offsets=None, table=None)) == ok
    assert calls(cache(), seqs(), width=0)[2] == binding.Q8_OK


_NO_DEVICE = r"""
import sys
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, sys.argv[2])
import test_cache_abi as t
print(*t.calls(t.cache(), t.seqs()), t.binding.q8_last_hip_error())
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
    *statuses, hip_err = [int(x) for x in res.stdout.split()]
    assert all(s in (binding.Q8_ERR_HIP, binding.Q8_ERR_UNSUPPORTED_DEVICE) for s in statuses), statuses


# ------------------------------------------------------------------ the binding

def tensors(pages=3, heads=2, page=16, dim=64):
    return (torch.zeros((pages, heads, page, dim), dtype=torch.int8),
            torch.zeros((pages, heads, page, dim // 32)),
            torch.zeros((pages, heads, page, dim), dtype=torch.int8),
            torch.zeros((pages, heads, page, dim // 32)))


def test_cache_handle_checks_its_tensors():
    k, ks, v, vs = tensors()
    with pytest.raises(TypeError):
        binding.Q8Cache(None, ks, v, vs)
    with pytest.raises(ValueError, match="rank 4"):
        binding.Q8Cache(k[0], ks, v, vs)
    with pytest.raises(ValueError, match="dim must be"):
        binding.Q8Cache(*tensors(dim=32))
    with pytest.raises(ValueError, match="page_size"):
        binding.Q8Cache(*tensors(page=24))
    with pytest.raises(ValueError, match="device tensor"):
        binding.Q8Cache(k, ks, v, vs)
    with pytest.raises(ValueError, match="torch.int8"):
        binding.Q8Cache(k.to(torch.uint8), ks, v, vs)


def test_row_tensors_are_checked():
    class Fake:
        device, dim, heads = torch.device("cpu"), 64, 2
    good = torch.zeros((5, 2, 64))
    assert binding._cache_rows("k", good, 5, 2, Fake) [0] == 128
    wide = torch.zeros((5, 300))[:, 3:131].unflatten(1, (2, 64))
    assert binding._cache_rows("k", wide, 5, 2, Fake)[0] == 300
    assert binding._cache_rows("k", good[:0], 0, 2, Fake)[0] == 128
    with pytest.raises(TypeError):
        binding._cache_rows("k", [1], None, 2, Fake)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        binding._cache_rows("k", good.double(), None, 2, Fake)
    with pytest.raises(ValueError, match="torch.float32"):
        binding._cache_rows("k", good.half(), None, 2, Fake, torch.float32)
    with pytest.raises(ValueError, match="shape"):
        binding._cache_rows("k", good, 4, 2, Fake)
    with pytest.raises(ValueError, match="shape"):
        binding._cache_rows("k", good, 5, 3, Fake)
    with pytest.raises(ValueError, match="dense"):
        binding._cache_rows("k", torch.zeros((5, 64, 2)).transpose(1, 2), 5, 2, Fake)
    with pytest.raises(ValueError, match="dense"):
        binding._cache_rows("k", torch.zeros((5, 2, 128))[..., ::2], 5, 2, Fake)
    with pytest.raises(ValueError, match="overlap"):
        binding._cache_rows("k", torch.zeros(64 * 8).as_strided((5, 2, 64), (64, 64, 1)), 5, 2, Fake)


def test_overlapping_row_tensors_are_refused():
    wide = torch.zeros((4, 400), dtype=torch.bfloat16)
    a, b = (wide[:, i:i + 128].unflatten(1, (2, 64)) for i in (1, 129))
    binding._check_apart("k", a, (("v", b), ("none", None)))
    binding._check_apart("k", b, (("v", a),))
    for i in (0, 2, 128):
        with pytest.raises(ValueError, match="overlaps"):
            binding._check_apart("k", a, (("v", wide[:, i:i + 128].unflatten(1, (2, 64))),))
    with pytest.raises(ValueError, match="overlaps"):      # another distance between rows
        binding._check_apart("k", a, (("v", wide.flatten()[129:129 + 2 * 128].unflatten(0, (2, 2, 64))),))
    # behind a's last row, and in the row below b's first byte
    binding._check_apart("k", a[:2], (("v", wide[2:, :128].unflatten(1, (2, 64))),))


def test_sequences_are_checked():
    class Fake(binding.Q8Cache):
        def __init__(self):
            self.device = torch.device("cpu")
    c, i32 = Fake(), torch.int32
    table, lengths, offsets = torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    s = binding._cache_seqs(c, table, lengths, offsets)
    assert (s.seqs, s.max_pages, s.table_stride) == (2, 3, 3)
    assert binding._cache_seqs(c, torch.zeros((2, 9), dtype=i32)[:, 2:5], lengths, offsets).table_stride == 9
    with pytest.raises(TypeError):
        binding._cache_seqs(None, table, lengths, offsets)
    with pytest.raises(TypeError):
        binding._cache_seqs(c, [[1]], lengths, offsets)
    with pytest.raises(ValueError, match="int32"):
        binding._cache_seqs(c, table.long(), lengths, offsets)
    with pytest.raises(ValueError, match="rank 1"):
        binding._cache_seqs(c, table, table, offsets)
    with pytest.raises(ValueError, match="offsets"):
        binding._cache_seqs(c, table, lengths, lengths)
    with pytest.raises(ValueError, match="contiguous"):
        binding._cache_seqs(c, table, torch.zeros(4, dtype=i32)[::2], offsets)
    with pytest.raises(ValueError, match="overlap"):
        binding._cache_seqs(c, torch.zeros(4, dtype=i32).as_strided((2, 3), (1, 1)), lengths, offsets)


def test_attention_holds_its_workspace_until_the_call_returns(monkeypatch):
    """The library enqueues two kernels that use it; freed before, another
    thread's allocation on the same stream could get the same memory in between."""
    import weakref
    made, seen = [], []
    empty = binding._empty_on

    def tracked(*args):
        t = empty(*args)
        made.append((weakref.ref(t), t.dtype, t.data_ptr()))
        return t

    def call(cache, stream, what, fn, *args):
        for ref, dtype, at in made:
            if dtype is torch.uint8:
                seen.append((ref() is not None, at in args))

    monkeypatch.setattr(binding, "_empty_on", tracked)
    monkeypatch.setattr(binding, "_call", call)
    monkeypatch.setattr(binding, "_attention_workspace", lambda *args: 4096)
    c = object.__new__(binding.Q8Cache)
    c.device, c.heads, c.dim, c.page_size, c.pages = torch.device("cpu"), 2, 64, 16, 3
    c._struct, c._spans = cache(), ()
    i32 = torch.int32
    q = torch.zeros((5, 4, 64))
    out = binding.q8_cache_attention(q, c, torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32),
                                     torch.zeros(3, dtype=i32))
    assert out.shape == q.shape
    assert seen == [(True, True)]


def test_attention_refuses_heads_that_do_not_fit():
    """A cache of no heads among them."""
    c = object.__new__(binding.Q8Cache)
    c.device, c.dim, c.page_size, c.pages = torch.device("cpu"), 64, 16, 3
    i32 = torch.int32
    held = torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    for c.heads, q_heads in ((2, 3), (2, 0), (4, 2), (0, 4), (0, 0)):
        with pytest.raises(ValueError, match="multiple"):
            binding.q8_cache_attention(torch.zeros((5, q_heads, 64)), c, *held)


def test_a_stream_of_another_device_is_refused():
    """Before anything is allocated or enqueued on it."""
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    c = object.__new__(binding.Q8Cache)
    c.device, c.heads, c.dim, c.page_size, c.pages = torch.device("cuda", 0), 2, 64, 16, 3
    rows, held = torch.zeros((5, 2, 64)), (torch.zeros((2, 3), dtype=torch.int32),) * 3
    for call in (lambda: binding.q8_cache_write(c, rows, rows, *held, stream=Stream()),
                 lambda: binding.q8_cache_read(c, *held, 5, stream=Stream()),
                 lambda: binding.q8_cache_keep(c, *held, held[0], stream=Stream()),
                 lambda: binding.q8_cache_attention(rows, c, *held, stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()
