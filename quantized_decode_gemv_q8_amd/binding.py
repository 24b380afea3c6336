"""Thin Python binding of libq8gemv.so (include/q8_gemv.h).

Argument marshalling only: every step of the computation runs in the HIP
library.  torch supplies device memory and the stream.  If the library is not
built this module raises; there is no fallback implementation.
"""

import ctypes
import os

import torch

from .build import LIB_PATH

Q8_OK = 0
Q8_ERR_INVALID = 1
Q8_ERR_TOO_LARGE = 2
Q8_ERR_UNSUPPORTED_DEVICE = 3
Q8_ERR_HIP = 4

BLOCK = 32
MAX_SIBLINGS = 4
PLAN_STREAM = 1
PLAN_MATRIX = 2

#: Every symbol include/q8_gemv.h declares.
EXPORTED = (
    "q8_matvec",
    "q8_matvec_noalloc",
    "q8_matvec_with_plan",
    "q8_matvec_choose_plan",
    "q8_matvec_fused",
    "q8_dot_t",
    "q8_dot_f32",
    "q8_dot_t_f32",
    "q8_cache_write",
    "q8_cache_read",
    "q8_cache_keep",
    "q8_cache_attention_workspace",
    "q8_cache_attention",
    "q8_status_string",
    "q8_last_hip_error",
    "q8_release",
)


class Q8Plan(ctypes.Structure):
    _fields_ = [("vec", ctypes.c_int32), ("m_tile", ctypes.c_int32),
                ("workgroups", ctypes.c_int32), ("waves", ctypes.c_int32), ("kind", ctypes.c_int32)]

    def as_dict(self):
        return {"vec": self.vec, "m_tile": self.m_tile, "workgroups": self.workgroups, "waves": self.waves,
                "kind": self.kind}


class Q8Sibling(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("S", ctypes.c_void_p), ("C", ctypes.c_void_p)]


class Q8Epilogue(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("corr", ctypes.c_void_p)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("KS", ctypes.c_void_p), ("V", ctypes.c_void_p), ("VS", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dim", ctypes.c_int32)]


class _SeqsStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64)]


class Q8Error(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = f"{what}: {q8_status_string(status)}"
        if status == Q8_ERR_HIP:
            msg += f" (hipError {q8_last_hip_error()})"
        super().__init__(msg)


_lib = None


def load():
    """The loaded library (ctypes.CDLL), loading it on first use."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m quantized_decode_gemv_q8_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.q8_matvec.argtypes = [p, p, p, p, i64, i64, i64, p]
    L.q8_matvec.restype = ctypes.c_int
    L.q8_matvec_noalloc.argtypes = [p, p, p, p, i64, i64, i64, p]
    L.q8_matvec_noalloc.restype = ctypes.c_int
    L.q8_matvec_with_plan.argtypes = [p, p, p, p, i64, i64, i64, ctypes.POINTER(Q8Plan), p]
    L.q8_matvec_with_plan.restype = ctypes.c_int
    L.q8_matvec_choose_plan.argtypes = [i64, i64, i64, i64, i64, i32, ctypes.POINTER(Q8Plan)]
    L.q8_matvec_choose_plan.restype = ctypes.c_int
    L.q8_matvec_fused.argtypes = [p, ctypes.POINTER(Q8Sibling), i32, i64, i64, i64,
                                  ctypes.POINTER(Q8Epilogue), ctypes.POINTER(Q8Plan), p]
    L.q8_matvec_fused.restype = ctypes.c_int
    L.q8_dot_t.argtypes = [p, p, p, i64, i64, i64, p]
    L.q8_dot_t.restype = ctypes.c_int
    for name in ("q8_dot_f32", "q8_dot_t_f32"):
        fn = getattr(L, name)
        fn.argtypes = [p, p, p, i64, i64, i64, ctypes.POINTER(Q8Epilogue), p]
        fn.restype = ctypes.c_int
    cache, seqs = ctypes.POINTER(_CacheStruct), ctypes.POINTER(_SeqsStruct)
    for name in ("q8_cache_write", "q8_cache_read"):
        fn = getattr(L, name)
        fn.argtypes = [cache, p, p, ctypes.c_int, i64, i64, i64, seqs, p]
        fn.restype = ctypes.c_int
    L.q8_cache_keep.argtypes = [cache, i64, seqs, p, i64, p]
    L.q8_cache_keep.restype = ctypes.c_int
    L.q8_cache_attention_workspace.argtypes = [cache, ctypes.c_int, i64, i32, seqs, ctypes.POINTER(i64)]
    L.q8_cache_attention_workspace.restype = ctypes.c_int
    L.q8_cache_attention.argtypes = [cache, p, p, ctypes.c_int, i64, i32, i64, i64, seqs, p, i64, ctypes.c_float,
                                     p, i64, p]
    L.q8_cache_attention.restype = ctypes.c_int
    L.q8_status_string.argtypes = [ctypes.c_int]
    L.q8_status_string.restype = ctypes.c_char_p
    L.q8_last_hip_error.argtypes = []
    L.q8_last_hip_error.restype = ctypes.c_int
    L.q8_release.argtypes = []
    L.q8_release.restype = None
    _lib = L
    return L


def q8_status_string(status):
    return load().q8_status_string(int(status)).decode()


def q8_last_hip_error():
    return load().q8_last_hip_error()


def q8_release():
    load().q8_release()


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check_tensor(name, t, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (dense row-major)")


def _check_disjoint(out_name, out, others):
    """The library requires outputs that share no bytes with any other
    argument; an overlap would be a silent race, so it is refused here."""
    if out.numel() == 0:
        return
    a0 = out.data_ptr()
    a1 = a0 + out.numel() * out.element_size()
    for name, t in others:
        if t is None or t.numel() == 0:
            continue
        b0 = t.data_ptr()
        b1 = b0 + t.numel() * t.element_size()
        if a0 < b1 and b0 < a1:
            raise ValueError(f"{out_name} overlaps {name}")


def _rank2(**named):
    for name, t in named.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 2:
            raise ValueError(f"{name} must be rank 2, got {t.dim()} dimensions")


def _q8_args(A, W, S, out):
    _rank2(A=A, W=W)
    M, K = A.shape
    N = W.shape[1]
    KB = (K + BLOCK - 1) // BLOCK
    _check_tensor("A", A, torch.float32, (M, K))
    _check_tensor("W", W, torch.int8, (K, N))
    _check_tensor("S", S, torch.float32, (KB, N))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check_tensor("out", out, torch.float32, (M, N))
    for t in (W, S, out):
        if t.device != A.device:
            raise ValueError("all tensors must be on one device")
    _check_disjoint("out", out, (("A", A), ("W", W), ("S", S)))
    return M, K, N, out


def q8_matvec(A, W, S, out=None, stream=None):
    """C[m,n] = sum_k A[m,k] W[k,n] S[k//32,n] on the GPU; returns C (f32 [M,N])."""
    M, K, N, out = _q8_args(A, W, S, out)
    with torch.cuda.device(A.device):
        st = load().q8_matvec(A.data_ptr(), W.data_ptr(), S.data_ptr(), out.data_ptr(),
                              M, K, N, _stream_handle(stream, A.device))
    if st != Q8_OK:
        raise Q8Error(st, "q8_matvec")
    return out


def q8_matvec_noalloc(A, W, S, out=None, stream=None):
    """q8_matvec through the library's fixed scratch array instead of its
    workspace: the call allocates nothing on the device (out must be given to
    avoid torch's allocation).  Calls that overlap in time on one device race."""
    M, K, N, out = _q8_args(A, W, S, out)
    with torch.cuda.device(A.device):
        st = load().q8_matvec_noalloc(A.data_ptr(), W.data_ptr(), S.data_ptr(), out.data_ptr(),
                                      M, K, N, _stream_handle(stream, A.device))
    if st != Q8_OK:
        raise Q8Error(st, "q8_matvec_noalloc")
    return out


def q8_matvec_with_plan(A, W, S, plan, out=None, stream=None):
    """q8_matvec with an explicit launch plan (dict with vec, m_tile, workgroups, waves, kind)."""
    M, K, N, out = _q8_args(A, W, S, out)
    pl = _plan_struct(plan)
    with torch.cuda.device(A.device):
        st = load().q8_matvec_with_plan(A.data_ptr(), W.data_ptr(), S.data_ptr(), out.data_ptr(),
                                        M, K, N, ctypes.byref(pl), _stream_handle(stream, A.device))
    if st != Q8_OK:
        raise Q8Error(st, "q8_matvec_with_plan")
    return out


def _plan_struct(plan):
    return Q8Plan(int(plan.get("vec", 0)), int(plan.get("m_tile", 0)),
                  int(plan.get("workgroups", 0)), int(plan.get("waves", 0)), int(plan.get("kind", 0)))


def q8_matvec_fused(A, Ws, Ss, outs=None, alpha=1.0, corr=None, plan=None, stream=None):
    """Sibling projections sharing A, in one launch, through the epilogue
    C_g = alpha * (A x dequant(W_g, S_g)) + corr[m] * C_g (corr: f32 [M] or
    None).  With corr the existing contents of outs are read.  Returns the
    list of C_g (f32 [M,N])."""
    if not isinstance(Ws, (list, tuple)) or not isinstance(Ss, (list, tuple)) or len(Ws) != len(Ss):
        raise ValueError("Ws and Ss must be lists of equal length")
    n = len(Ws)
    if not 1 <= n <= MAX_SIBLINGS:
        raise ValueError(f"1..{MAX_SIBLINGS} siblings, got {n}")
    if outs is None:
        if corr is not None:
            raise ValueError("corr reads the existing outputs: pass outs")
        outs = [None] * n
    if len(outs) != n:
        raise ValueError("outs must have one entry per sibling")
    res = []
    M = K = N = None
    for W, S, out in zip(Ws, Ss, outs):
        M, K, N, out = _q8_args(A, W, S, out)
        res.append(out)
    if corr is not None:
        _check_tensor("corr", corr, torch.float32, (M,))
        if corr.device != A.device:
            raise ValueError("all tensors must be on one device")
    inputs = [("corr", corr)] + [(f"Ws[{j}]", W) for j, W in enumerate(Ws)] + \
        [(f"Ss[{j}]", S) for j, S in enumerate(Ss)]
    for g, C in enumerate(res):
        _check_disjoint(f"outs[{g}]", C, inputs + [(f"outs[{j}]", res[j]) for j in range(g)])
    sib = (Q8Sibling * n)(*[Q8Sibling(W.data_ptr(), S.data_ptr(), C.data_ptr()) for W, S, C in zip(Ws, Ss, res)])
    ep = Q8Epilogue(float(alpha), corr.data_ptr() if corr is not None else None)
    pl = ctypes.byref(_plan_struct(plan)) if plan is not None else None
    with torch.cuda.device(A.device):
        st = load().q8_matvec_fused(A.data_ptr(), sib, n, M, K, N, ctypes.byref(ep), pl,
                                    _stream_handle(stream, A.device))
    if st != Q8_OK:
        raise Q8Error(st, "q8_matvec_fused")
    return res


def q8_matvec_choose_plan(M, K, N, w_align=256, s_align=256, num_cus=256):
    """The plan q8_matvec would pick (host logic only; touches no device)."""
    pl = Q8Plan()
    st = load().q8_matvec_choose_plan(int(M), int(K), int(N), int(w_align), int(s_align),
                                      int(num_cus), ctypes.byref(pl))
    if st != Q8_OK:
        raise Q8Error(st, "q8_matvec_choose_plan")
    return pl.as_dict()


def q8_dot_t(A, W, out=None, stream=None):
    """C[m,n] = sum_k A[m,k] W[n,k] in exact i32 on the GPU; returns C (i32 [M,N])."""
    _rank2(A=A, W=W)
    M, K = A.shape
    N = W.shape[0]
    _check_tensor("A", A, torch.int8, (M, K))
    _check_tensor("W", W, torch.int8, (N, K))
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32, device=A.device)
    _check_tensor("out", out, torch.int32, (M, N))
    if W.device != A.device or out.device != A.device:
        raise ValueError("all tensors must be on one device")
    _check_disjoint("out", out, (("A", A), ("W", W)))
    with torch.cuda.device(A.device):
        st = load().q8_dot_t(A.data_ptr(), W.data_ptr(), out.data_ptr(), M, K, N,
                             _stream_handle(stream, A.device))
    if st != Q8_OK:
        raise Q8Error(st, "q8_dot_t")
    return out


def _dense(name, A, B, transposed, out, alpha, corr, stream):
    _rank2(A=A, B=B)
    M, K = A.shape
    N = B.shape[0] if transposed else B.shape[1]
    _check_tensor("A", A, torch.float32, (M, K))
    _check_tensor("B", B, torch.float32, (N, K) if transposed else (K, N))
    if out is None:
        if corr is not None:
            raise ValueError("corr reads the existing output: pass out")
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check_tensor("out", out, torch.float32, (M, N))
    if corr is not None:
        _check_tensor("corr", corr, torch.float32, (M,))
    for t in (B, out) + ((corr,) if corr is not None else ()):
        if t.device != A.device:
            raise ValueError("all tensors must be on one device")
    _check_disjoint("out", out, (("A", A), ("B", B), ("corr", corr)))
    ep = Q8Epilogue(float(alpha), corr.data_ptr() if corr is not None else None)
    with torch.cuda.device(A.device):
        st = getattr(load(), name)(A.data_ptr(), B.data_ptr(), out.data_ptr(), M, K, N, ctypes.byref(ep),
                                   _stream_handle(stream, A.device))
    if st != Q8_OK:
        raise Q8Error(st, name)
    return out


def q8_dot_f32(A, B, out=None, alpha=1.0, corr=None, stream=None):
    """C = alpha * (A @ B) (+ corr[m] * C) for f32 A [M,K], B [K,N]; returns C (f32 [M,N])."""
    return _dense("q8_dot_f32", A, B, False, out, alpha, corr, stream)


def q8_dot_t_f32(A, B, out=None, alpha=1.0, corr=None, stream=None):
    """C = alpha * (A @ B^T) (+ corr[m] * C) for f32 A [M,K], B [N,K]; returns C (f32 [M,N])."""
    return _dense("q8_dot_t_f32", A, B, True, out, alpha, corr, stream)


# ------------------------------------------------------------------ the Q8_0 cache

#: Element types of the rows outside the cache.
_ROW_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class Q8Cache:
    """Keys and values of an attention layer in pages, in Q8_0.

    k, v              i8  [pages, heads, page_size, dim], codes
    k_scale, v_scale  f32 [pages, heads, page_size, dim // 32]

    A token's value is code * scale.  Codes of a row lie in pair order: the
    natural order [dim // 32, 16, 2] is stored as [16, dim // 32, 2].  The tensors
    stay the caller's; the handle only checks them once.
    """

    __slots__ = ("k", "k_scale", "v", "v_scale", "pages", "heads", "page_size", "dim", "device", "_struct", "_spans")

    def __init__(self, k, k_scale, v, v_scale):
        if not isinstance(k, torch.Tensor):
            raise TypeError("k must be a torch.Tensor")
        if k.dim() != 4:
            raise ValueError(f"k must be rank 4, got {k.dim()} dimensions")
        codes = k.shape
        pages, heads, page_size, dim = codes
        if dim not in (64, 128, 256):
            raise ValueError(f"dim must be 64, 128 or 256, got {dim}")
        if page_size not in (16, 32, 64, 128, 256, 512, 1024):
            raise ValueError(f"page_size must be a power of two from 16 to 1024, got {page_size}")
        scales, device = (pages, heads, page_size, dim // BLOCK), k.device
        for name, t, dtype, shape in (("k", k, torch.int8, codes), ("k_scale", k_scale, torch.float32, scales),
                                      ("v", v, torch.int8, codes), ("v_scale", v_scale, torch.float32, scales)):
            _check_tensor(name, t, dtype, shape)
            if t.get_device() != device.index:
                raise ValueError("all tensors must be on one device")
        self.k, self.k_scale, self.v, self.v_scale = k, k_scale, v, v_scale
        self.pages, self.heads, self.page_size, self.dim, self.device = pages, heads, page_size, dim, device
        n = pages * heads * page_size * dim
        a, b, c, d = at = k.data_ptr(), k_scale.data_ptr(), v.data_ptr(), v_scale.data_ptr()
        self._spans = (a, a + n), (b, b + n // 8), (c, c + n), (d, d + n // 8)
        edge = 0
        for a, b in sorted(self._spans):
            if a < edge and n:
                raise ValueError("the cache's tensors overlap")
            edge = b
        self._struct = _CacheStruct(*at, pages, heads, page_size, dim)

    def _apart(self, name, a, b):
        """Refuses a tensor of a call (bytes a .. b - 1) that shares any with the cache."""
        for c, d in self._spans:
            if a < d and c < b:
                raise ValueError(f"{name} overlaps the cache")

    @classmethod
    def empty(cls, pages, heads, page_size, dim, device="cuda"):
        """A cache with new tensors; what it holds is undefined until it is written."""
        def new(last, dtype):
            return torch.empty((pages, heads, page_size, last), dtype=dtype, device=device)
        return cls(new(dim, torch.int8), new(dim // BLOCK, torch.float32),
                   new(dim, torch.int8), new(dim // BLOCK, torch.float32))


def _cache_seqs(cache, table, lengths, offsets, stream=None):
    """The checked descriptor of a call's sequences; the call's stream is checked too."""
    if not isinstance(cache, Q8Cache):
        raise TypeError("cache must be a Q8Cache")
    if stream is not None and stream.device != cache.device:
        raise ValueError(f"the stream is of {stream.device}, the cache of {cache.device}")
    index, i32 = cache.device.index, torch.int32
    for name, t, rank in (("table", table, 2), ("lengths", lengths, 1), ("offsets", offsets, 1)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not i32:
            raise ValueError(f"{name} must be torch.int32, got {t.dtype}")
        if t.get_device() != index and t.device != cache.device:
            raise ValueError("all tensors must be on one device")
        if t.dim() != rank:
            raise ValueError(f"{name} must be rank {rank}, got {t.dim()} dimensions")
        if not t.is_contiguous() and t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
    n, pages = table.shape
    if lengths.shape[0] != n or offsets.shape[0] != n + 1:
        raise ValueError(f"{n} rows of table need {n} lengths and {n + 1} offsets, got "
                         f"{lengths.shape[0]} and {offsets.shape[0]}")
    stride = table.stride(0) if n > 1 else pages
    if stride < pages:
        raise ValueError("rows of table must not overlap")
    return _SeqsStruct(table.data_ptr(), lengths.data_ptr(), offsets.data_ptr(), n, pages, stride)


def _seqs_spans(seqs):
    """Names and bytes of a descriptor's tensors."""
    n, t, l, o = seqs.seqs, seqs.table or 0, seqs.lengths or 0, seqs.offsets or 0
    return (("table", t, t + 4 * ((n - 1) * seqs.table_stride + seqs.max_pages) if n else t),
            ("lengths", l, l + 4 * n), ("offsets", o, o + 4 * n + 4))


def _cache_rows(name, t, rows, heads, cache, dtype=None):
    """Checks a row tensor [rows, heads, dim]: rows may be apart, a row is dense.
    Returns its row stride and the address of its first byte."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _ROW_TYPES or (dtype is not None and t.dtype != dtype):
        want = dtype if dtype is not None else "float32, bfloat16 or float16"
        raise ValueError(f"{name} must be {want}, got {t.dtype}")
    if t.get_device() != cache.device.index and t.device != cache.device:
        raise ValueError("all tensors must be on one device")
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.dim or (rows is not None and shape[0] != rows) or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape ({'rows' if rows is None else rows}, "
                         f"{'heads' if heads is None else heads}, {cache.dim}), got {tuple(shape)}")
    n, h, dim = shape
    if n == 0 or h == 0 or t.is_contiguous():
        return h * dim, t.data_ptr()
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and s1 != dim):
        raise ValueError(f"{name} must be dense in its last two dimensions")
    if n > 1 and s0 < h * dim:
        raise ValueError(f"rows of {name} must not overlap")
    return s0, t.data_ptr()


def _span(t):
    """First byte and one past the last byte of a tensor with non-negative strides."""
    if t.numel() == 0:
        return 0, 0
    a = t.data_ptr()
    if t.is_contiguous():
        return a, a + t.numel() * t.element_size()
    return a, a + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _check_apart(out_name, out, others):
    """_check_disjoint for row tensors, whose rows may be apart."""
    a0, a1 = _span(out)
    for name, t in others:
        if t is None:
            continue
        b0, b1 = _span(t)
        if a0 < b1 and b0 < a1 and not _interleaved(out, t):
            raise ValueError(f"{out_name} overlaps {name}")


def _interleaved(a, b):
    """Whether two row tensors are views of one wide one, side by side: rows
    equally far apart, and apart from each other within that distance."""
    if a.dim() != 3 or b.dim() != 3:
        return False
    pitch = a.stride(0) * a.element_size()
    if pitch == 0 or pitch != b.stride(0) * b.element_size():
        return False
    between = (b.data_ptr() - a.data_ptr()) % pitch
    return between >= _span(a[0])[1] - _span(a[0])[0] and pitch - between >= _span(b[0])[1] - _span(b[0])[0]


def _empty_on(stream, shape, dtype, device):
    """A new tensor whose memory is ordered with the work of `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(cache, stream, what, fn, *args):
    """fn(*args, stream) on the cache's device; an error status raises."""
    device = cache.device
    if torch.cuda.current_device() == device.index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, _stream_handle(stream, device))
    if st != Q8_OK:
        raise Q8Error(st, what)


def q8_cache_write(cache, k, v, table, lengths, offsets, stream=None):
    """Quantises rows k and v ([rows, heads, dim]) into the cache: sequence b's
    newest offsets[b+1] - offsets[b] tokens of lengths[b] are rows offsets[b]
    .. of k and v, and live in the pages table[b]."""
    seqs = _cache_seqs(cache, table, lengths, offsets, stream)
    ks, k0 = _cache_rows("k", k, None, cache.heads, cache)
    vs, v0 = _cache_rows("v", v, k.shape[0], cache.heads, cache, k.dtype)
    rows, size = k.shape[0], k.element_size()
    width = cache.heads * cache.dim
    if rows:
        cache._apart("k", k0, k0 + ((rows - 1) * ks + width) * size)
        cache._apart("v", v0, v0 + ((rows - 1) * vs + width) * size)
    for name, a, b in _seqs_spans(seqs):
        cache._apart(name, a, b)
    _call(cache, stream, "q8_cache_write", load().q8_cache_write, cache._struct, k0, v0, _ROW_TYPES[k.dtype], rows, ks,
          vs, seqs)


def q8_cache_read(cache, table, lengths, offsets, rows, dtype=torch.float32, k=None, v=None, stream=None):
    """The newest offsets[b+1] - offsets[b] tokens of each sequence as rows
    [rows, heads, dim] of dtype; returns (k, v).  Rows of no sequence keep what
    the given k and v hold (new tensors: undefined)."""
    seqs = _cache_seqs(cache, table, lengths, offsets, stream)
    rows = int(rows)
    shape = (rows, cache.heads, cache.dim)
    if k is None and v is None:
        if dtype not in _ROW_TYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        k, v = _empty_on(stream, (2,) + shape, dtype, cache.device).unbind()
        ks = vs = cache.heads * cache.dim
        k0, v0 = k.data_ptr(), v.data_ptr()
    elif k is None or v is None:
        raise ValueError("pass both k and v, or neither")
    else:
        ks, k0 = _cache_rows("k", k, rows, cache.heads, cache)
        vs, v0 = _cache_rows("v", v, rows, cache.heads, cache, k.dtype)
        inputs = (("table", table), ("lengths", lengths), ("offsets", offsets))
        cache._apart("k", *_span(k))
        cache._apart("v", *_span(v))
        _check_apart("k", k, inputs)
        _check_apart("v", v, inputs + (("k", k),))
    _call(cache, stream, "q8_cache_read", load().q8_cache_read, cache._struct, k0, v0, _ROW_TYPES[k.dtype], rows, ks, vs,
          seqs)
    return k, v


def q8_cache_keep(cache, table, lengths, offsets, keep, stream=None, rows=None):
    """Moves new token keep[b, a] of sequence b to the place of its new token a,
    a = 0, 1, ...; keep is i32 [sequences, width], strictly ascending until its
    first negative entry.  rows: of the row tensors that the offsets refer to; a
    sequence whose offsets pass them has no new tokens, as in q8_cache_write
    (None: offsets may be of any size)."""
    seqs = _cache_seqs(cache, table, lengths, offsets, stream)
    if not isinstance(keep, torch.Tensor):
        raise TypeError("keep must be a torch.Tensor")
    if keep.dim() != 2:
        raise ValueError(f"keep must be rank 2, got {keep.dim()} dimensions")
    _check_tensor("keep", keep, torch.int32, (table.shape[0], keep.shape[1]))
    if keep.device != cache.device:
        raise ValueError("all tensors must be on one device")
    cache._apart("keep", *_span(keep))
    for name, a, b in _seqs_spans(seqs):
        cache._apart(name, a, b)
    _call(cache, stream, "q8_cache_keep", load().q8_cache_keep, cache._struct,
          MAX_CACHE_ROWS if rows is None else int(rows), seqs, keep.data_ptr(), keep.shape[1])


#: Most rows a call's offsets may refer to.
MAX_CACHE_ROWS = (1 << 31) - 1


def q8_cache_attention(q, cache, table, lengths, offsets, tree=None, alpha=None, out=None, stream=None):
    """Attention of the new tokens' queries q ([rows, q_heads, dim]) over the
    cache, their own keys and values included; returns out, shaped like q.

    Row offsets[b] + i (new token i of sequence b) sees every token before the
    new ones and, of the new ones, those up to i; or with tree (i64 [rows, words])
    those j whose bit j % 64 of word j // 64 of the row is set.  alpha: scale of
    the scores, 1 / sqrt(dim) if None.  Rows of no sequence keep what out holds
    (a new out: undefined); rows that see nothing are zeros.
    """
    seqs = _cache_seqs(cache, table, lengths, offsets, stream)
    qs, q0 = _cache_rows("q", q, None, None, cache)
    rows, q_heads = q.shape[0], q.shape[1]
    if q_heads == 0 or cache.heads == 0 or q_heads % cache.heads:
        raise ValueError(f"the heads of q must be a multiple of the cache's {cache.heads}, got {q_heads}")
    words = 0
    if tree is not None:
        if not isinstance(tree, torch.Tensor):
            raise TypeError("tree must be a torch.Tensor")
        if tree.dim() != 2:
            raise ValueError(f"tree must be rank 2, got {tree.dim()} dimensions")
        words = tree.shape[1]
        _check_tensor("tree", tree, torch.int64, (rows, words))
        if tree.device != cache.device:
            raise ValueError("all tensors must be on one device")
    if alpha is None:
        alpha = cache.dim ** -0.5
    if out is None:
        out = _empty_on(stream, (rows, q_heads, cache.dim), q.dtype, cache.device)
        os_, out0 = q_heads * cache.dim, out.data_ptr()
    else:
        os_, out0 = _cache_rows("out", out, rows, q_heads, cache, q.dtype)
        cache._apart("out", *_span(out))
        _check_apart("out", out, (("q", q), ("table", table), ("lengths", lengths), ("offsets", offsets),
                                  ("tree", tree)))
    need = _attention_workspace(cache, _ROW_TYPES[q.dtype], rows, q_heads, seqs)
    # Held until both of the call's kernels are enqueued: what the same stream's
    # next owner of the memory enqueues then comes after them.
    work = _empty_on(stream, (need,), torch.uint8, cache.device) if need else None
    mask = None
    if tree is not None:  # an empty tree still is one: no new token is seen
        mask = tree.data_ptr() if words and rows else offsets.data_ptr() & -8
    _call(cache, stream, "q8_cache_attention", load().q8_cache_attention, cache._struct, q0, out0,
          _ROW_TYPES[q.dtype], rows, q_heads, qs, os_, seqs, mask, words, float(alpha),
          None if work is None else work.data_ptr(), need)
    return out


#: Workspace sizes by the extents that they follow from.
_WORKSPACE = {}


def _attention_workspace(cache, type_, rows, q_heads, seqs):
    # whether there are any pages counts: without, no token of the table is one
    key = (cache.device.index, cache.pages > 0, cache.heads, cache.page_size, cache.dim, type_, rows, q_heads,
           seqs.seqs, seqs.max_pages)
    need = _WORKSPACE.get(key)
    if need is None:
        size = ctypes.c_int64(0)
        with torch.cuda.device(cache.device):
            st = load().q8_cache_attention_workspace(cache._struct, type_, rows, q_heads, seqs, size)
        if st != Q8_OK:
            raise Q8Error(st, "q8_cache_attention")
        if len(_WORKSPACE) >= 4096:
            _WORKSPACE.clear()
        need = _WORKSPACE[key] = size.value
    return need
