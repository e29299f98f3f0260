"""Thin Python binding of libfp8q's C ABI (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of the method: it turns torch tensors into device pointers, the
current torch stream into a ``cudaStream_t`` and a non-zero status into an
exception.  There is no CPU path: if ``libfp8q.so`` is missing or no GPU is
usable the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfp8q.so")

E4M3, E5M2, E2M1 = 0, 1, 2
MX_FLOOR, MX_CEIL, MX_NEAREST = 0, 1, 2
MX_ROWWISE, MX_COLWISE = 0, 1
EST_MAX_WINDOW, EST_SMOOTHED = 0, 1
F32, BF16 = 0, 1
NO_EXP = -(2 ** 31)
MAX_WINDOW = 256
WORKSPACE_ZEROED = 16384      # MX_KV_WORKSPACE_ZEROED

_STATUS = {0: "FP8Q_OK", -1: "FP8Q_EINVAL", -2: "FP8Q_EALIGN", -3: "FP8Q_EDTYPE", -4: "FP8Q_ECUDA",
           -5: "FP8Q_EHANDLE", -6: "FP8Q_ENOMEM", -7: "FP8Q_EDEVICE", -8: "FP8Q_ESIZE"}


class Fp8qError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        msg = f"{what} failed: {_STATUS.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


_lib = None


def load() -> ctypes.CDLL:
    """Load libfp8q.so (built by ``__graft_entry__.build()`` or
    ``tensor_scaling_cast_gb300.build``).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run tensor_scaling_cast_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    p, i, i64, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    L.fp8q_create.argtypes = [i, i, i, i, ctypes.POINTER(p)]
    L.fp8q_create_ex.argtypes = [i, i, i, i, i, f, i, ctypes.POINTER(p)]
    L.fp8q_get_estimator_state.argtypes = [p, ctypes.POINTER(f), ctypes.POINTER(i),
                                           ctypes.POINTER(ctypes.c_longlong)]
    L.fp8q_set_estimator_state.argtypes = [p, f, i, ctypes.c_longlong]
    L.fp8q_destroy.argtypes = [p]
    L.fp8q_cast.argtypes = [p, p, i, i64, p, p, p, p, p]
    L.fp8q_cast_multi.argtypes = [p, p, p, p, p, p, p, p, i, p]
    L.fp8q_cast_multi_ex.argtypes = [p, p, p, p, p, p, p, p, p, p, i, p]
    L.fp8q_loss_scaler_create.argtypes = [f, i, f, f, ctypes.POINTER(p)]
    L.fp8q_loss_scaler_destroy.argtypes = [p]
    L.fp8q_loss_scaler_update.argtypes = [p, p, i, p, p, p]
    L.fp8q_loss_scaler_read.argtypes = [p, ctypes.POINTER(f), ctypes.POINTER(i)]
    L.mx_cast.argtypes = [p, i, i64, i64, i, i, p, p, p, p]
    L.mx_cast_ex.argtypes = [p, i, i64, i64, i, i, i, i, p, p, p, p]
    L.mx_cast_dual.argtypes = [p, i, i64, i64, i, i, i, p, p, p, p, p, p, p]
    L.fp8q_cast_transpose.argtypes = [p, p, i, i64, i64, p, p, p, p, p, p]
    L.fp8q_amax_history.argtypes = [p, ctypes.POINTER(f), i, ctypes.POINTER(i)]
    L.fp8q_scale_state.argtypes = [p, ctypes.POINTER(i), ctypes.POINTER(ctypes.c_longlong)]
    L.fp8q_set_history.argtypes = [p, ctypes.POINTER(f), i, i]
    L.fp8q_reset.argtypes = [p]
    L.fp8q_error_stats.argtypes = [p, i, i64, p, i, p, p, p]
    L.mx_error_stats.argtypes = [p, i, i64, i64, p, p, i, p, p]
    L.fp8q_error_stats_noalloc.argtypes = [p, i, i64, p, i, p, p, p]
    L.mx_kv_write.argtypes = [p, p, p, i, i64, i64, i64, i64, i64, p, i, p]
    L.mx_kv_read.argtypes = [p, p, i64, p, p, i, i64, i64, i64, i64, p]
    L.mx_kv_attention.argtypes = [p, p, i, i64, i, i64, i64, p, i64, i64, p, p, p, p, i64, i, i, i, f, i, p,
                                  i64, p]
    L.mx_kv_attention_workspace.argtypes = [p, i64, i, i, i, i]
    L.mx_kv_attention_workspace.restype = i64
    L.fp8q_pipeline_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    L.fp8q_pipeline_status.restype = i
    L.fp8q_pipeline_selftest.argtypes = [p]
    L.fp8q_pipeline_selftest.restype = i
    L.fp8q_strerror.argtypes = [i]
    L.fp8q_strerror.restype = ctypes.c_char_p
    L.fp8q_last_cuda_error.restype = ctypes.c_char_p
    L.fp8q_launch_count.restype = ctypes.c_longlong
    for name in ("mx_cast_dual", "fp8q_cast_transpose", "fp8q_cast_multi_ex", "fp8q_loss_scaler_create", "fp8q_loss_scaler_destroy",
                 "fp8q_loss_scaler_update", "fp8q_loss_scaler_read",
                 "fp8q_create", "fp8q_create_ex", "fp8q_get_estimator_state",
                 "fp8q_set_estimator_state", "fp8q_destroy", "fp8q_cast", "fp8q_cast_multi", "mx_cast", "mx_cast_ex",
                 "fp8q_amax_history", "fp8q_scale_state", "fp8q_set_history", "fp8q_reset",
                 "fp8q_error_stats", "mx_error_stats", "fp8q_error_stats_noalloc",
                 "mx_kv_write", "mx_kv_read", "mx_kv_attention"):
        getattr(L, name).restype = i
    _lib = L
    return L


def _check(status: int, what: str):
    if status != 0:
        detail = ""
        if status == -4:
            detail = load().fp8q_last_cuda_error().decode()
        raise Fp8qError(status, what, detail)


# The entry points declare their pointer arguments as c_void_p, so plain
# Python ints (and None for NULL) are passed straight through.
def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported input dtype {t.dtype}: bf16 or fp32")


# torch's raw getter of the current stream (the public path builds a Stream
# object per call); falls back to the public path where it is absent.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def fp8q_pipeline_status() -> int:
    """Pipeline waits that timed out on the current device since the last call."""
    n = ctypes.c_uint()
    _check(load().fp8q_pipeline_status(ctypes.byref(n)), "fp8q_pipeline_status")
    return n.value


def fp8q_pipeline_selftest(stream=None):
    """Launch the never-completed barrier wait (see the C header)."""
    _check(load().fp8q_pipeline_selftest(_stream(stream)), "fp8q_pipeline_selftest")


def launch_count() -> int:
    return int(load().fp8q_launch_count())


# ---- handles ---------------------------------------------------------------

def fp8q_create(fmt: int, window: int, margin: int = 0, hysteresis: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(load().fp8q_create(fmt, window, margin, hysteresis, ctypes.byref(h)), "fp8q_create")
    return h.value


def fp8q_create_ex(fmt: int, window: int, margin: int = 0, hysteresis: int = 0,
                   estimator: int = EST_MAX_WINDOW, alpha: float = 1.0, interval: int = 1) -> int:
    h = ctypes.c_void_p()
    _check(load().fp8q_create_ex(fmt, window, margin, hysteresis, estimator, alpha, interval,
                                 ctypes.byref(h)), "fp8q_create_ex")
    return h.value


def fp8q_get_estimator_state(h: int):
    """(running average or None, number of casts)."""
    a, ha, st = ctypes.c_float(), ctypes.c_int(), ctypes.c_longlong()
    _check(load().fp8q_get_estimator_state(h, ctypes.byref(a), ctypes.byref(ha),
                                           ctypes.byref(st)), "fp8q_get_estimator_state")
    return (a.value if ha.value else None), st.value


def fp8q_set_estimator_state(h: int, average, steps: int):
    _check(load().fp8q_set_estimator_state(h, 0.0 if average is None else average,
                                           0 if average is None else 1, steps),
           "fp8q_set_estimator_state")


def fp8q_destroy(h: int):
    _check(load().fp8q_destroy(h), "fp8q_destroy")


def fp8q_cast(h: int, x: torch.Tensor, q: torch.Tensor, scale_inv=None, amax=None, clipped=None,
              stream=None):
    """x: contiguous bf16/fp32 CUDA tensor; q: uint8 CUDA tensor of x.numel()
    bytes; scale_inv / amax: float32 CUDA scalars; clipped: int64 CUDA scalar
    (read as uint64)."""
    _check(load().fp8q_cast(h, _ptr(x), _dtype(x), x.numel(), _ptr(q),
                            _ptr(scale_inv), _ptr(amax), _ptr(clipped), _stream(stream)),
           "fp8q_cast")


def fp8q_cast_multi(hs, xs, qs, scale_inv=None, amax=None, clipped=None, stream=None):
    """hs: handles; xs / qs: lists of CUDA tensors; scale_inv / amax: float32
    CUDA tensors [count]; clipped: int64 CUDA tensor [count]."""
    n = len(hs)
    H = (ctypes.c_void_p * n)(*hs)
    X = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
    Q = (ctypes.c_void_p * n)(*[q.data_ptr() for q in qs])
    D = (ctypes.c_int * n)(*[_dtype(x) for x in xs])
    N = (ctypes.c_int64 * n)(*[x.numel() for x in xs])
    _check(load().fp8q_cast_multi(H, X, D, N, Q, _ptr(scale_inv), _ptr(amax), _ptr(clipped), n,
                                  _stream(stream)), "fp8q_cast_multi")


def fp8q_cast_multi_ex(hs, xs, qs, scale_inv=None, amax=None, clipped=None, nonfinite=None,
                       underflow=None, stream=None):
    """fp8q_cast_multi plus int64 CUDA tensors [count] of non-finite and
    underflow counts (either may be None)."""
    n = len(hs)
    H = (ctypes.c_void_p * n)(*hs)
    X = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
    Q = (ctypes.c_void_p * n)(*[q.data_ptr() for q in qs])
    D = (ctypes.c_int * n)(*[_dtype(x) for x in xs])
    N = (ctypes.c_int64 * n)(*[x.numel() for x in xs])
    _check(load().fp8q_cast_multi_ex(H, X, D, N, Q, _ptr(scale_inv), _ptr(amax), _ptr(clipped),
                                     _ptr(nonfinite), _ptr(underflow), n, _stream(stream)),
           "fp8q_cast_multi_ex")


def fp8q_loss_scaler_create(init_scale: float, growth_interval: int, min_scale: float = 1.0,
                            max_scale: float = 2.0 ** 24) -> int:
    h = ctypes.c_void_p()
    _check(load().fp8q_loss_scaler_create(init_scale, growth_interval, min_scale, max_scale,
                                          ctypes.byref(h)), "fp8q_loss_scaler_create")
    return h.value


def fp8q_loss_scaler_destroy(h: int):
    _check(load().fp8q_loss_scaler_destroy(h), "fp8q_loss_scaler_destroy")


def fp8q_loss_scaler_update(h: int, nonfinite: torch.Tensor, scale=None, skip=None, stream=None):
    """nonfinite: int64 CUDA tensor of counts; scale: float32 CUDA scalar;
    skip: int32 CUDA scalar."""
    _check(load().fp8q_loss_scaler_update(h, _ptr(nonfinite), nonfinite.numel(),
                                          _ptr(scale), _ptr(skip), _stream(stream)),
           "fp8q_loss_scaler_update")


def fp8q_loss_scaler_read(h: int):
    """(scale, clean-step streak)."""
    sc, g = ctypes.c_float(), ctypes.c_int()
    _check(load().fp8q_loss_scaler_read(h, ctypes.byref(sc), ctypes.byref(g)),
           "fp8q_loss_scaler_read")
    return sc.value, g.value


def mx_cast(x: torch.Tensor, fmt: int, headroom: int, q: torch.Tensor, e8m0: torch.Tensor,
            clipped=None, stream=None):
    rows, cols = x.shape
    _check(load().mx_cast(_ptr(x), _dtype(x), rows, cols, fmt, headroom, _ptr(q), _ptr(e8m0),
                          _ptr(clipped), _stream(stream)), "mx_cast")


def mx_cast_ex(x: torch.Tensor, fmt: int, rule: int, headroom: int, axis: int, q: torch.Tensor,
               e8m0: torch.Tensor, clipped=None, stream=None):
    """axis MX_ROWWISE: e8m0 [rows, cols/32]; MX_COLWISE: e8m0 [rows/32, cols]."""
    rows, cols = x.shape
    _check(load().mx_cast_ex(_ptr(x), _dtype(x), rows, cols, fmt, rule, headroom, axis, _ptr(q),
                             _ptr(e8m0), _ptr(clipped), _stream(stream)), "mx_cast_ex")


def mx_cast_dual(x: torch.Tensor, fmt: int, rule: int, headroom: int, q_row, e8_row, q_colt, e8_colt,
                 clipped_row=None, clipped_col=None, stream=None):
    """Row-wise MX of x and row-wise MX of x^T (column-wise blocks written
    transposed) from one read: q_row [rows, cols], e8_row [rows, cols/32],
    q_colt [cols, rows], e8_colt [cols, rows/32]."""
    rows, cols = x.shape
    _check(load().mx_cast_dual(_ptr(x), _dtype(x), rows, cols, fmt, rule, headroom, _ptr(q_row),
                               _ptr(e8_row), _ptr(q_colt), _ptr(e8_colt), _ptr(clipped_row),
                               _ptr(clipped_col), _stream(stream)), "mx_cast_dual")


def fp8q_cast_transpose(h: int, x: torch.Tensor, q, qt, scale_inv=None, amax=None, clipped=None,
                        stream=None):
    """Per-tensor cast of x [rows, cols] to q [rows, cols] and qt [cols, rows]."""
    rows, cols = x.shape
    _check(load().fp8q_cast_transpose(h, _ptr(x), _dtype(x), rows, cols, _ptr(q),
                                      _ptr(qt), _ptr(scale_inv), _ptr(amax), _ptr(clipped),
                                      _stream(stream)), "fp8q_cast_transpose")


def fp8q_amax_history(h: int, capacity: int = MAX_WINDOW) -> list[float]:
    buf = (ctypes.c_float * max(1, capacity))()
    nv = ctypes.c_int()
    _check(load().fp8q_amax_history(h, buf, capacity, ctypes.byref(nv)),
           "fp8q_amax_history")
    return [buf[i] for i in range(nv.value)]


def fp8q_scale_state(h: int):
    """(previous exponent or None, number of casts)."""
    e = ctypes.c_int()
    st = ctypes.c_longlong()
    _check(load().fp8q_scale_state(h, ctypes.byref(e), ctypes.byref(st)),
           "fp8q_scale_state")
    return (None if e.value == NO_EXP else e.value), st.value


def fp8q_set_history(h: int, values, prev_exp=None):
    buf = (ctypes.c_float * max(1, len(values)))(*values)
    _check(load().fp8q_set_history(h, buf, len(values),
                                   NO_EXP if prev_exp is None else int(prev_exp)),
           "fp8q_set_history")


def fp8q_reset(h: int):
    _check(load().fp8q_reset(h), "fp8q_reset")


def fp8q_error_stats(x: torch.Tensor, q: torch.Tensor, fmt: int, scale_inv: torch.Tensor,
                     out: torch.Tensor, stream=None):
    _check(load().fp8q_error_stats(_ptr(x), _dtype(x), x.numel(), _ptr(q), fmt, _ptr(scale_inv),
                                   _ptr(out), _stream(stream)), "fp8q_error_stats")


def fp8q_error_stats_noalloc(x: torch.Tensor, q: torch.Tensor, fmt: int, scale_inv: torch.Tensor,
                             out: torch.Tensor, stream=None):
    """fp8q_error_stats without any device allocation (fixed library
    scratch; n <= 2^32; calls must not overlap on the GPU)."""
    _check(load().fp8q_error_stats_noalloc(_ptr(x), _dtype(x), x.numel(), _ptr(q), fmt,
                                           _ptr(scale_inv), _ptr(out), _stream(stream)),
           "fp8q_error_stats_noalloc")


def mx_error_stats(x: torch.Tensor, q: torch.Tensor, e8m0: torch.Tensor, fmt: int,
                   out: torch.Tensor, stream=None):
    rows, cols = x.shape
    _check(load().mx_error_stats(_ptr(x), _dtype(x), rows, cols, _ptr(q), _ptr(e8m0), fmt,
                                 _ptr(out), _stream(stream)), "mx_error_stats")


# ---- key/value cache ---------------------------------------------------------

class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_q", ctypes.c_void_p), ("k_e8m0", ctypes.c_void_p), ("v_q", ctypes.c_void_p),
                ("v_e8m0", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class MXKVCache:
    """The four arrays of a paged key/value cache and their description for
    the C calls: codes uint8 [pages, kv_heads, page_size, head_dim / 2 (E2M1)
    or head_dim] and E8M0 bytes uint8 [pages, kv_heads, page_size,
    head_dim / 32], for keys and for values."""

    def __init__(self, k_q: torch.Tensor, k_e8m0: torch.Tensor, v_q: torch.Tensor, v_e8m0: torch.Tensor,
                 fmt: int = E2M1):
        pages, heads, page, blocks = k_e8m0.shape
        dim = 32 * blocks
        row = (pages, heads, page, dim // 2 if fmt == E2M1 else dim)
        for t, shape in ((k_q, row), (v_q, row), (k_e8m0, k_e8m0.shape), (v_e8m0, k_e8m0.shape)):
            if t.dtype != torch.uint8 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
                raise TypeError(f"cache arrays are contiguous uint8 of shape {tuple(shape)}: "
                                f"got {t.dtype} {tuple(t.shape)}")
        self.k_q, self.k_e8m0, self.v_q, self.v_e8m0 = k_q, k_e8m0, v_q, v_e8m0
        self.fmt, self.num_pages, self.kv_heads, self.page_size, self.head_dim = fmt, pages, heads, page, dim
        self._struct = _KVCacheStruct(k_q.data_ptr(), k_e8m0.data_ptr(), v_q.data_ptr(), v_e8m0.data_ptr(),
                                      pages, page, heads, dim, fmt)
        self._ref = ctypes.addressof(self._struct)
        self._scale = dim ** -0.5

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: int = E2M1,
                 device="cuda") -> "MXKVCache":
        """A cache of zeroed arrays."""
        row = head_dim // 2 if fmt == E2M1 else head_dim
        q, e = (num_pages, kv_heads, page_size, row), (num_pages, kv_heads, page_size, head_dim // 32)
        return cls(*(torch.zeros(s, dtype=torch.uint8, device=device) for s in (q, e, q, e)), fmt=fmt)


# Few-token calls are bound by the host: the checks read each shape and stride
# once, and the entry points' results are what is left to check.
def _kv_pair(cache, k, v, slots, what):
    """(tokens, dtype code, strides of k and v) of a write's or read's rows."""
    shape, ks, vs, dtype = k.shape, k.stride(), v.stride(), k.dtype
    if (len(ks) != 3 or shape != v.shape or shape[2] != cache.head_dim or shape[1] != cache.kv_heads
            or ks[2] != 1 or vs[2] != 1 or v.dtype is not dtype or slots.dtype is not torch.int64
            or slots.numel() != shape[0] or not slots.is_contiguous()):
        raise TypeError(f"{what}: k and v alike, [tokens, {cache.kv_heads}, {cache.head_dim}] with consecutive "
                        f"elements, and contiguous int64 slots, one per token: got {tuple(shape)}, "
                        f"{tuple(v.shape)} with strides {ks}, {vs}, slots {slots.dtype} {tuple(slots.shape)}")
    return shape[0], BF16 if dtype is torch.bfloat16 else _dtype(k), ks, vs


def mx_kv_write(cache: MXKVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, rule: int = MX_FLOOR,
                stream=None):
    """Quantise k and v [tokens, kv_heads, head_dim] (bf16 or fp32, any token and
    head stride) into the cache slots `slots` (int64; negative: not written)."""
    n, dtype, ks, vs = _kv_pair(cache, k, v, slots, "mx_kv_write")
    st = (_lib or load()).mx_kv_write(cache._ref, k.data_ptr(), v.data_ptr(), dtype, n, ks[0], ks[1], vs[0], vs[1],
                                      slots.data_ptr(), rule, _stream(stream))
    if st:
        _check(st, "mx_kv_write")


def mx_kv_read(cache: MXKVCache, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None):
    """Read the slots back into k and v [tokens, kv_heads, head_dim] (bf16 or
    fp32); a negative slot gives zeros."""
    n, dtype, ks, vs = _kv_pair(cache, k, v, slots, "mx_kv_read")
    st = (_lib or load()).mx_kv_read(cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), dtype, ks[0],
                                     ks[1], vs[0], vs[1], _stream(stream))
    if st:
        _check(st, "mx_kv_read")


def mx_kv_attention_workspace(cache: MXKVCache, q: torch.Tensor, page_table: torch.Tensor, max_q=None):
    """A workspace for mx_kv_attention calls of these shapes, ready for its first
    use, or None where they need none.  max_q None: enough whatever max_q those
    calls have or leave out; with the call's own it can be far smaller (decode
    steps: 1).  One per stream; it serves every call whose own shapes ask for no
    more bytes."""
    total, q_heads = q.shape[0], q.shape[1]
    # the plans differ by rows per key/value head: up to 8, 16, 24, 32, and more
    group = max(1, q_heads // cache.kv_heads)
    bounds = [max_q] if max_q is not None else [max(1, r) for r in (8 // group, 16 // group, 24 // group, 32 // group, total)]
    sizes = [load().mx_kv_attention_workspace(cache._ref, total, q_heads, page_table.shape[0], m, page_table.shape[1])
             for m in bounds]
    n = min(sizes) if min(sizes) < 0 else max(sizes)
    if n < 0:
        _check(n, "mx_kv_attention_workspace")
    if not n:
        return None
    ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    ws[:WORKSPACE_ZEROED].zero_()
    return ws


def mx_kv_attention(cache: MXKVCache, q: torch.Tensor, out: torch.Tensor, page_table: torch.Tensor,
                    kv_lens: torch.Tensor, cu_q=None, max_q=None, scale=None, window: int = 0, lse=None,
                    workspace=None, stream=None):
    """Attention of q [total_q, q_heads, head_dim] (bf16) over the 4-bit cache,
    into out of the same shape.  page_table int32 [batch, pages], kv_lens int32
    [batch], cu_q int32 [batch + 1] (None: one query per sequence), max_q >= the
    queries of any sequence (None: 1 without cu_q, total_q with it; the closer
    the bound, the better the plan), scale (None: head_dim ** -0.5), lse
    float32 [total_q, q_heads] or None, workspace of mx_kv_attention_workspace
    for the same max_q, or without one."""
    shape, qs, os_ = q.shape, q.stride(), out.stride()
    table, ts = page_table.shape, page_table.stride()
    if (len(shape) != 3 or shape[2] != cache.head_dim or out.shape != shape or qs[2] != 1 or os_[2] != 1
            or q.dtype is not torch.bfloat16 or out.dtype is not torch.bfloat16):
        raise TypeError(f"mx_kv_attention: q and out are bf16 [total_q, q_heads, {cache.head_dim}] with consecutive "
                        f"elements: got {q.dtype} {tuple(shape)}, {out.dtype} {tuple(out.shape)}, strides {qs}, {os_}")
    if (page_table.dtype is not torch.int32 or len(table) != 2 or (ts[1] != 1 and table[1] > 1)
            or kv_lens.dtype is not torch.int32 or kv_lens.numel() != table[0] or not kv_lens.is_contiguous()
            or (cu_q is not None and (cu_q.dtype is not torch.int32 or cu_q.numel() != table[0] + 1
                                      or not cu_q.is_contiguous()))
            or (lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:2]
                                     or not lse.is_contiguous()))):
        raise TypeError("mx_kv_attention: page_table int32 [batch, pages], kv_lens int32 [batch], "
                        "cu_q int32 [batch + 1], lse float32 [total_q, q_heads]")
    if max_q is None:
        max_q = 1 if cu_q is None else max(1, shape[0])
    st = (_lib or load()).mx_kv_attention(
        cache._ref, q.data_ptr(), BF16, shape[0], shape[1], qs[0], qs[1], out.data_ptr(), os_[0], os_[1],
        None if lse is None else lse.data_ptr(), None if cu_q is None else cu_q.data_ptr(), kv_lens.data_ptr(),
        page_table.data_ptr(), ts[0], table[1], table[0], max_q, cache._scale if scale is None else scale, window,
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
        _stream(stream))
    if st:
        _check(st, "mx_kv_attention")


# ---- convenience wrapper ---------------------------------------------------

class ScaledCast:
    """One tensor's scaling state on the GPU (owns an fp8q handle) with
    output buffers allocated by torch."""

    def __init__(self, fmt: int, window: int, margin: int = 0, hysteresis: int = 0,
                 estimator: int = EST_MAX_WINDOW, alpha: float = 1.0, interval: int = 1):
        self.fmt, self.window, self.margin, self.hysteresis = fmt, window, margin, hysteresis
        self.handle = fp8q_create_ex(fmt, window, margin, hysteresis, estimator, alpha, interval)

    def __call__(self, x: torch.Tensor, q: torch.Tensor | None = None, stream=None):
        """Returns (q uint8, scale_inv f32[1], amax f32[1], clipped i64[1]) on x's device."""
        dev = x.device
        if q is None:
            q = torch.empty(x.shape, dtype=torch.uint8, device=dev)
        # one 16-byte allocation: scale_inv f32, amax f32, clipped i64
        outs = torch.empty(4, dtype=torch.float32, device=dev)
        scale_inv, amax, clipped = outs[0:1], outs[1:2], outs[2:4].view(torch.int64)
        fp8q_cast(self.handle, x, q, scale_inv, amax, clipped, stream)
        return q, scale_inv, amax, clipped

    def history(self):
        return fp8q_amax_history(self.handle, max(1, self.window))

    def state(self):
        return fp8q_scale_state(self.handle)

    def set_history(self, values, prev_exp=None):
        fp8q_set_history(self.handle, values, prev_exp)

    def reset(self):
        fp8q_reset(self.handle)

    def close(self):
        if self.handle:
            fp8q_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
