"""ctypes binding of libq8proj.so: argument marshalling only.

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it checks tensor dtypes/shapes/devices, passes raw
device pointers, sizes and the current CUDA stream, and turns a non-zero
status into :class:`Q8Error`.  If the library is missing the call fails
loudly; there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading
from array import array

from . import build as _build

_lock = threading.Lock()
_lib = None

STATUS_NAMES = {0: "Q8_OK", 1: "Q8_ERR_ARG", 2: "Q8_ERR_ALIGN", 3: "Q8_ERR_DEVICE", 4: "Q8_ERR_LAUNCH",
                5: "Q8_ERR_DEVICE_TIMEOUT", 6: "Q8_ERR_CUDA", 7: "Q8_ERR_TOO_BIG", 8: "Q8_ERR_DATA"}

# (name, restype, argtypes) of every symbol include/q8proj.h declares.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
SIGNATURES = {
    "q8_plane_rows": (_I64, [_I64]),
    "q8_strerror": (ctypes.c_char_p, [_INT]),
    "quantize_q8_0": (_INT, [_P, _I64, _I64, _P, _P, _I64, _P]),
    "rmsnorm_quant": (_INT, [_P, _P, ctypes.c_float, _P, _I64, _I64, _P, _P, _I64, _P]),
    "swiglu_quant": (_INT, [_P, _P, _P, _I64, _I64, _P, _P, _I64, _P]),
    "q8_0_gemv": (_INT, [_P, _I64, _I64, _P, _P, _P, _P]),
    "q8_0_gemm_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "q8_0_gemm": (_INT, [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, ctypes.c_size_t, _P]),
    "q8_0_gemm_prepared_weights_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "q8_0_gemm_prepare_weights": (_INT, [_P, _I64, _I64, _P, ctypes.c_size_t, _P]),
    "q8_0_gemm_prepared_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "q8_0_gemm_prepared": (_INT, [_P, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, ctypes.c_size_t, _P]),
    "q8_0_gemm_mma": (_INT, [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P]),
    "q8_0_gemm_noalloc": (_INT, [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P]),
    "q8_0_gemm_noalloc_max_bytes": (ctypes.c_size_t, []),
    "q8_0_gemv_grouped": (_INT, [_P, _INT, _I64, _P, _P, _P]),
    "q8_0_gemv_fused": (_INT, [_P, _INT, _I64, _INT, _P, _P, _P, ctypes.c_float, _P]),
    "q8_0_gemv_gate_up": (_INT, [_P, _P, _I64, _I64, _P, _P, _INT, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P]),
    "q8_0_gemv_batched": (_INT, [_P, _I64, _I64, _P, _P, _I64, _P, _P]),
    "q8_0_gemv_batched_grouped": (_INT, [_P, _INT, _I64, _P, _P, _I64, _P]),
    "q4a_gemv": (_INT, [_P, _I64, _I64, _P, _P, _P, _P]),
    "q4a_gemv_batched": (_INT, [_P, _I64, _I64, _P, _P, _I64, _P, _P]),
    "q4a_gemv_batched_grouped": (_INT, [_P, _INT, _I64, _P, _P, _I64, _P]),
    "q8_kv_plan": (_INT, [_P, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P]),
    "q8_kv_append": (_INT, [_P, _I64, _P, _P, _P, _I64, _P]),
    "q8_tree_attention_workspace_bytes": (ctypes.c_size_t, [_P, _I64, _I64]),
    "q8_tree_attention_needs_workspace": (_INT, [_P, _I64, _I64, _I64, _I64]),
    "q8_tree_attention": (_INT, [_P, _I64, _P, _I64, ctypes.c_float, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _P,
                                 _P, _P, ctypes.c_size_t, _P]),
    "q8_kv_accept": (_INT, [_P, _P, _I64, _P, _P, _I64, _P, _P, _I64, _P, _P]),
    "q8_moe_route_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "q8_moe_route": (_INT, [_P, _I64, _I64, _I64, _INT, ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "q8_0_experts_gemm_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "q8_0_experts_gemm": (_INT, [_P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _P, _P, ctypes.c_size_t, _P]),
    "q8_0_experts_gate_up_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I64, _I64, _I64]),
    "q8_0_experts_gate_up": (_INT, [_P, _P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P, ctypes.c_size_t,
                                    _P]),
    "rmsnorm_residual_quant": (_INT, [_P, ctypes.c_float, _P, _P, _I64, _P, _P, _I64, _P, ctypes.c_float, _P, _I64, _P,
                                      ctypes.c_float, _P, _P, _I64, _I64, _P, _P, _I64, _P]),
    "q8_check": (_INT, [_P]),
    "q8_num_sms": (_INT, []),
}


MAX_GROUP = 8
KV_F16, KV_INT8 = 1, 2
TREE_MAX_NODES = 64
KV_MAX_BATCH = 4096
GEMV_MAX_TOKENS = 16
ROUTE_CHOSEN, ROUTE_ALL = 1, 2
MAX_EXPERTS = 1024
MAX_TOP_K = 16
PRODUCER_QUANT, PRODUCER_RMSNORM, PRODUCER_SWIGLU = 1, 2, 3


class GemvProj(ctypes.Structure):
    """C struct q8_gemv_proj: one projection of a grouped GEMV."""

    _fields_ = [("w", ctypes.c_void_p), ("n", ctypes.c_int64), ("y", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    """C struct q8_kv_cache."""

    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("layers", _I64), ("n_pages", _I64),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class KvCache:
    """A paged key/value cache: the caller's tensors and the descriptor the calls take.

    ``k``, ``v``: f16, or int8 codes, [layers][n_pages][kv_heads][page_size][head_dim]; ``k_scale``,
    ``v_scale``: f32 [layers][n_pages][kv_heads][page_size], with int8 only.  :func:`empty_kv_cache` makes one.
    The descriptor has the tensors' addresses and sizes as they were given, so none of them can be replaced."""

    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_kv_heads", "_page_size", "_head_dim", "_dev", "_ref", "_words")
    k, v, k_scale, v_scale, kv_heads, page_size, head_dim, dev, ref = (
        property(operator.attrgetter("_" + name))
        for name in ("k", "v", "k_scale", "v_scale", "kv_heads", "page_size", "head_dim", "dev", "ref"))

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch

        shape, dt = k.shape, k.dtype
        if len(shape) != 5 or v.shape != shape:
            raise ValueError("k, v: expected two [layers][n_pages][kv_heads][page_size][head_dim] tensors")
        int8 = dt is torch.int8
        if not int8 and dt is not torch.float16:
            raise ValueError(f"k: expected float16 or int8, got {dt}")
        if int8 != (k_scale is not None) or int8 != (v_scale is not None):
            raise ValueError("k_scale and v_scale with int8, and only then")
        dev = self._dev = k.get_device()
        kp, vp = _beside(k, dt, dev, "k"), _beside(v, dt, dev, "v")
        ks = vs = 0
        if int8:
            if k_scale.shape != shape[:-1] or v_scale.shape != shape[:-1]:
                raise ValueError("k_scale, v_scale: expected [layers][n_pages][kv_heads][page_size]")
            ks = _beside(k_scale, torch.float32, dev, "k_scale")
            vs = _beside(v_scale, torch.float32, dev, "v_scale")
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        layers, n_pages, self._kv_heads, self._page_size, self._head_dim = shape
        # a KvCacheDesc's bytes (a Structure takes several times as long to make); sizes past 32 bits are refused below
        if max(shape[2:]) >= 1 << 31:
            raise ValueError("k: kv_heads, page_size and head_dim have 32 bits")
        self._words = array("q", (kp, vp, ks, vs, layers, n_pages, shape[2] | shape[3] << 32,
                                  shape[4] | (KV_INT8 if int8 else KV_F16) << 32))
        self._ref = self._words.buffer_info()[0]


class Q8Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib().q8_strerror(status).decode() if _lib is not None else ""
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}: {msg}")


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libq8proj.so (built in-tree by ``build.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libq8proj.so is not built ({path}); run int8_quantized_projection_gb300.build")
            h = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(h, name)
                f.restype = res
                f.argtypes = args
            _lib = h
        return _lib


def load():
    return lib()


def _stream(stream):
    if stream is None:
        import torch

        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _check(fn, st):
    if st != 0:
        raise Q8Error(fn, st)


class Bound:
    """A C entry point with its arguments already marshalled.

    Calling it re-issues the same launch (same pointers, sizes and stream)
    with one ctypes call, which keeps the host cost of a decode step far below
    the GPU time of its kernels.  Returned by the ``bind=True`` form of every
    launching function."""

    __slots__ = ("name", "fn", "args", "_keep")

    def __init__(self, name, args):
        self.name = name
        self.fn = getattr(lib(), name)
        self.args = args
        self._keep = None

    def __call__(self):
        st = self.fn(*self.args)
        if st != 0:
            raise Q8Error(self.name, st)


def _launch(name, args, bind):
    if bind:
        return Bound(name, args)
    _check(name, getattr(lib(), name)(*args))
    return None


def _need(t, dtype, name):
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of {dtype}, got {t.dtype} on {t.device}")


def q8_plane_rows(rows: int) -> int:
    return int(lib().q8_plane_rows(rows))


def q8_num_sms() -> int:
    return int(lib().q8_num_sms())


def q8_check(stream=None) -> None:
    _check("q8_check", lib().q8_check(_stream(stream)))


def quantize_q8_0(x, qs, ds, stream=None, bind=False):
    """x f32 [rows][k] -> plane (qs int8 [rows_pad][k], ds int32 [rows_pad][k/32])."""
    import torch

    _need(x, torch.float32, "x"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds")
    rows, k = x.shape
    rows_pad = qs.shape[0]
    if qs.shape != (rows_pad, k) or ds.shape != (rows_pad, k // 32):
        raise ValueError("plane shape mismatch")
    return _launch("quantize_q8_0", (_ptr(x), rows, k, _ptr(qs), _ptr(ds), rows_pad, _stream(stream)), bind)


def rmsnorm_quant(x, w, eps: float, y, qs, ds, stream=None, bind=False):
    """``y=None``: mode 2, only the plane is written (the f32 output is dead)."""
    import torch

    for t, n in ((x, "x"), (w, "w")) + (((y, "y"),) if y is not None else ()):
        _need(t, torch.float32, n)
    _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds")
    rows, d = x.shape
    rows_pad = qs.shape[0]
    if ((y is not None and y.shape != x.shape) or w.shape != (d,) or qs.shape != (rows_pad, d)
            or ds.shape != (rows_pad, d // 32)):
        raise ValueError("shape mismatch")
    yp = _ptr(y) if y is not None else ctypes.c_void_p(0)
    return _launch("rmsnorm_quant", (_ptr(x), _ptr(w), ctypes.c_float(eps), yp, rows, d, _ptr(qs), _ptr(ds),
                                     rows_pad, _stream(stream)), bind)


def swiglu_quant(gate, up, y, qs, ds, stream=None, bind=False):
    """``y=None``: mode 2, only the plane is written (the f32 output is dead)."""
    import torch

    for t, n in ((gate, "gate"), (up, "up")) + (((y, "y"),) if y is not None else ()):
        _need(t, torch.float32, n)
    _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds")
    rows, nf = gate.shape
    rows_pad = qs.shape[0]
    if (up.shape != gate.shape or (y is not None and y.shape != gate.shape) or qs.shape != (rows_pad, nf)
            or ds.shape != (rows_pad, nf // 32)):
        raise ValueError("shape mismatch")
    yp = _ptr(y) if y is not None else ctypes.c_void_p(0)
    return _launch("swiglu_quant", (_ptr(gate), _ptr(up), yp, rows, nf, _ptr(qs), _ptr(ds), rows_pad,
                                    _stream(stream)), bind)


def q8_0_gemv(w, n: int, k: int, qs, ds, y, stream=None, bind=False):
    """w uint8 [n*k/32*34] Q8_0 blocks; plane row 0 of (qs, ds); y f32 [n]."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    if w.numel() != n * (k // 32) * 34 or y.numel() < n or qs.shape[-1] != k:
        raise ValueError("shape mismatch")
    return _launch("q8_0_gemv", (_ptr(w), n, k, _ptr(qs), _ptr(ds), _ptr(y), _stream(stream)), bind)


def q8_0_gemv_batched(w, n: int, k: int, qs, ds, t: int, y, stream=None, bind=False):
    """Y[t][n] f32 for plane rows [0, t), 1 <= t <= 16, weights read once for all t."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    if w.numel() != n * (k // 32) * 34 or y.numel() < t * n or qs.shape[-1] != k or qs.shape[0] < t:
        raise ValueError("shape mismatch")
    return _launch("q8_0_gemv_batched", (_ptr(w), n, k, _ptr(qs), _ptr(ds), t, _ptr(y), _stream(stream)), bind)


def q8_0_gemv_batched_grouped(projs, k: int, qs, ds, t: int, stream=None, bind=False):
    """Several small-batch projections of the same plane rows [0, t) in one launch.

    ``projs`` is a sequence of (w uint8 Q8_0 blocks, n, y f32 [t][n]) sharing k."""
    import torch

    _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds")
    if not 1 <= len(projs) <= MAX_GROUP or qs.shape[-1] != k or qs.shape[0] < t:
        raise ValueError("1..8 projections sharing k and the plane")
    arr = (GemvProj * len(projs))()
    keep = []
    for i, (w, n, y) in enumerate(projs):
        _need(w, torch.uint8, "w"), _need(y, torch.float32, "y")
        if w.numel() != n * (k // 32) * 34 or y.numel() < t * n:
            raise ValueError("shape mismatch")
        arr[i] = GemvProj(w.data_ptr(), n, y.data_ptr())
        keep.append((w, y))
    args = (ctypes.cast(arr, ctypes.c_void_p), len(projs), k, _ptr(qs), _ptr(ds), t, _stream(stream))
    if bind:
        b = Bound("q8_0_gemv_batched_grouped", args)
        b._keep = (arr, keep)  # the descriptor array must outlive the bound launch
        return b
    _check("q8_0_gemv_batched_grouped", lib().q8_0_gemv_batched_grouped(*args))
    return None


def q4a_gemv(w, n: int, k: int, qs, ds, y, stream=None, bind=False):
    """w uint8 [n*k/32*20] asymmetric 4-bit blocks; plane row 0 of (qs, ds); y f32 [n]."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    if w.numel() != n * (k // 32) * 20 or y.numel() < n or qs.shape[-1] != k:
        raise ValueError("shape mismatch")
    return _launch("q4a_gemv", (_ptr(w), n, k, _ptr(qs), _ptr(ds), _ptr(y), _stream(stream)), bind)


def q4a_gemv_batched(w, n: int, k: int, qs, ds, t: int, y, stream=None, bind=False):
    """Asymmetric 4-bit weights, Y[t][n] f32 for plane rows [0, t), 1 <= t <= 16, weights read once for all t."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    if w.numel() != n * (k // 32) * 20 or y.numel() < t * n or qs.shape[-1] != k or qs.shape[0] < t:
        raise ValueError("shape mismatch")
    return _launch("q4a_gemv_batched", (_ptr(w), n, k, _ptr(qs), _ptr(ds), t, _ptr(y), _stream(stream)), bind)


def q4a_gemv_batched_grouped(projs, k: int, qs, ds, t: int, stream=None, bind=False):
    """Several asymmetric 4-bit small-batch projections of the same plane rows [0, t) in one launch.

    ``projs`` is a sequence of (w uint8 20-byte blocks, n, y f32 [t][n]) sharing k."""
    import torch

    _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds")
    if not 1 <= len(projs) <= MAX_GROUP or qs.shape[-1] != k or qs.shape[0] < t:
        raise ValueError("1..8 projections sharing k and the plane")
    arr = (GemvProj * len(projs))()
    keep = []
    for i, (w, n, y) in enumerate(projs):
        _need(w, torch.uint8, "w"), _need(y, torch.float32, "y")
        if w.numel() != n * (k // 32) * 20 or y.numel() < t * n:
            raise ValueError("shape mismatch")
        arr[i] = GemvProj(w.data_ptr(), n, y.data_ptr())
        keep.append((w, y))
    args = (ctypes.cast(arr, ctypes.c_void_p), len(projs), k, _ptr(qs), _ptr(ds), t, _stream(stream))
    if bind:
        b = Bound("q4a_gemv_batched_grouped", args)
        b._keep = (arr, keep)  # the descriptor array must outlive the bound launch
        return b
    _check("q4a_gemv_batched_grouped", lib().q4a_gemv_batched_grouped(*args))
    return None


def q8_0_gemv_grouped(projs, k: int, qs, ds, stream=None, bind=False):
    """Several projections of one activation in one launch.

    ``projs`` is a sequence of (w uint8 Q8_0 blocks, n, y f32 [n]) sharing k and
    plane row 0 of (qs, ds)."""
    import torch

    _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds")
    if not 1 <= len(projs) <= MAX_GROUP or qs.shape[-1] != k:
        raise ValueError("1..8 projections sharing k")
    arr = (GemvProj * len(projs))()
    keep = []
    for i, (w, n, y) in enumerate(projs):
        _need(w, torch.uint8, "w"), _need(y, torch.float32, "y")
        if w.numel() != n * (k // 32) * 34 or y.numel() < n:
            raise ValueError("shape mismatch")
        arr[i] = GemvProj(w.data_ptr(), n, y.data_ptr())
        keep.append((w, y))
    args = (ctypes.cast(arr, ctypes.c_void_p), len(projs), k, _ptr(qs), _ptr(ds), _stream(stream))
    if bind:
        b = Bound("q8_0_gemv_grouped", args)
        b._keep = (arr, keep)  # the descriptor array must outlive the bound launch
        return b
    _check("q8_0_gemv_grouped", lib().q8_0_gemv_grouped(*args))
    return None


def _proj_array(projs, k):
    import torch

    if not 1 <= len(projs) <= MAX_GROUP:
        raise ValueError("1..8 projections sharing k")
    arr = (GemvProj * len(projs))()
    keep = []
    for i, (w, n, y) in enumerate(projs):
        _need(w, torch.uint8, "w"), _need(y, torch.float32, "y")
        if w.numel() != n * (k // 32) * 34 or y.numel() < n:
            raise ValueError("shape mismatch")
        arr[i] = GemvProj(w.data_ptr(), n, y.data_ptr())
        keep.append((w, y))
    return arr, keep


def q8_0_gemv_fused(projs, k: int, producer: int, a, b=None, norm_w=None, eps: float = 0.0, stream=None,
                    bind=False):
    """Grouped batch-1 projections whose activation the same launch produces.

    ``producer`` is PRODUCER_QUANT (a = x f32 [k]), PRODUCER_RMSNORM (a = x,
    norm_w = w f32 [k], eps) or PRODUCER_SWIGLU (a = gate, b = up, f32 [k]);
    ``projs`` as for :func:`q8_0_gemv_grouped`."""
    import torch

    for t, nm in ((a, "a"), (b, "b"), (norm_w, "norm_w")):
        if t is not None:
            _need(t, torch.float32, nm)
            if t.numel() < k:
                raise ValueError(f"{nm}: fewer than k elements")
    arr, keep = _proj_array(projs, k)
    nul = ctypes.c_void_p(0)
    args = (ctypes.cast(arr, ctypes.c_void_p), len(projs), k, int(producer), _ptr(a),
            _ptr(b) if b is not None else nul, _ptr(norm_w) if norm_w is not None else nul, float(eps),
            _stream(stream))
    if bind:
        bd = Bound("q8_0_gemv_fused", args)
        bd._keep = (arr, keep, a, b, norm_w)
        return bd
    _check("q8_0_gemv_fused", lib().q8_0_gemv_fused(*args))
    return None


def q8_0_gemv_gate_up(w_gate, w_up, nf: int, k: int, qs_out, ds_out, qs=None, ds=None, producer: int = 0, a=None,
                      norm_w=None, eps: float = 0.0, y_gate=None, y_up=None, stream=None, bind=False):
    """Gate and up projections of one token with SwiGLU + q8_0 quantize in the same launch.

    The activation is plane row 0 of (qs, ds) when ``producer`` is 0, else
    produced in the launch (PRODUCER_QUANT: a = x; PRODUCER_RMSNORM: a = x,
    norm_w, eps).  Writes plane row 0 of silu(gate) * up into (qs_out,
    ds_out); y_gate / y_up (f32 [nf]) are optional."""
    import torch

    _need(w_gate, torch.uint8, "w_gate"), _need(w_up, torch.uint8, "w_up")
    _need(qs_out, torch.int8, "qs_out"), _need(ds_out, torch.int32, "ds_out")
    if w_gate.numel() != nf * (k // 32) * 34 or w_up.numel() != w_gate.numel():
        raise ValueError("weight shape mismatch")
    if qs_out.shape[-1] != nf or ds_out.shape[-1] != nf // 32:
        raise ValueError("output plane shape mismatch")
    for t, nm, dt in ((qs, "qs", torch.int8), (ds, "ds", torch.int32), (a, "a", torch.float32),
                      (norm_w, "norm_w", torch.float32), (y_gate, "y_gate", torch.float32),
                      (y_up, "y_up", torch.float32)):
        if t is not None:
            _need(t, dt, nm)
    nul = ctypes.c_void_p(0)
    opt = lambda t: _ptr(t) if t is not None else nul  # noqa: E731
    args = (_ptr(w_gate), _ptr(w_up), nf, k, opt(qs), opt(ds), int(producer), opt(a), opt(norm_w), float(eps),
            opt(y_gate), opt(y_up), _ptr(qs_out), _ptr(ds_out), _stream(stream))
    return _launch("q8_0_gemv_gate_up", args, bind)


def q8_0_gemm_workspace_bytes(n: int, t: int, k: int) -> int:
    return int(lib().q8_0_gemm_workspace_bytes(n, t, k))


def gemm_workspace(n: int, t: int, k: int, device="cuda"):
    """Allocate (with PyTorch) the scratch q8_0_gemm needs for (t, k); None if it needs none."""
    import torch

    nbytes = q8_0_gemm_workspace_bytes(n, t, k)
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def q8_0_gemm_prepared_weights_bytes(n: int, k: int) -> int:
    return int(lib().q8_0_gemm_prepared_weights_bytes(n, k))


def q8_0_gemm_prepared_workspace_bytes(n: int, t: int, k: int) -> int:
    return int(lib().q8_0_gemm_prepared_workspace_bytes(n, t, k))


def q8_0_gemm_prepare_weights(w, n: int, k: int, wprep=None, stream=None):
    """Write the GEMM's prepared form of the Q8_0 matrix ``w`` (n x k) into
    ``wprep`` (a uint8 CUDA tensor of q8_0_gemm_prepared_weights_bytes(n, k)
    bytes; allocated here with PyTorch when None) and return it."""
    import torch

    _need(w, torch.uint8, "w")
    if w.numel() != n * (k // 32) * 34:
        raise ValueError("shape mismatch")
    nbytes = q8_0_gemm_prepared_weights_bytes(n, k)
    if nbytes == 0:
        raise ValueError("no prepared form for this shape ((k/32) % 8 != 0 or past the GEMM's limits)")
    if wprep is None:
        wprep = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    _need(wprep, torch.uint8, "wprep")
    _check("q8_0_gemm_prepare_weights",
           lib().q8_0_gemm_prepare_weights(_ptr(w), n, k, _ptr(wprep), wprep.numel(), _stream(stream)))
    return wprep


def q8_0_gemm_prepared(w, wprep, n: int, k: int, qs, ds, t: int, y, workspace=None, stream=None, bind=False):
    """q8_0_gemm whose tcgen05 path reads ``wprep`` (q8_0_gemm_prepare_weights's
    output) instead of widening ``w`` on every call; ``w`` serves the other
    paths (t <= 64, (k/32) % 8 != 0) and may be None when the call takes the
    tcgen05 path."""
    import torch

    _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    if w is not None:
        _need(w, torch.uint8, "w")
    if wprep is not None:
        _need(wprep, torch.uint8, "wprep")
    rows_pad = qs.shape[0]
    if y.numel() < t * n or qs.shape[-1] != k or ds.shape[0] != rows_pad:
        raise ValueError("shape mismatch")
    nbytes = q8_0_gemm_prepared_workspace_bytes(n, t, k)
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=y.device)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    nul = ctypes.c_void_p(0)
    args = (_ptr(w) if w is not None else nul, _ptr(wprep) if wprep is not None else nul, n, k, _ptr(qs), _ptr(ds),
            t, rows_pad, _ptr(y), _ptr(workspace) if workspace is not None else nul,
            workspace.numel() if workspace is not None else 0, _stream(stream))
    if bind:
        b = Bound("q8_0_gemm_prepared", args)
        b._keep = (workspace, w, wprep)
        return b
    _check("q8_0_gemm_prepared", lib().q8_0_gemm_prepared(*args))
    return None


def q8_0_gemm(w, n: int, k: int, qs, ds, t: int, y, workspace=None, stream=None, bind=False):
    """Y[t][n] f32 = plane rows [0, t) x Q8_0 weights.

    ``workspace`` is a uint8 CUDA tensor of at least q8_0_gemm_workspace_bytes(n, t, k)
    bytes; when None one is allocated here with PyTorch (the library never allocates)."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    rows_pad = qs.shape[0]
    if w.numel() != n * (k // 32) * 34 or y.numel() < t * n or qs.shape[-1] != k or ds.shape[0] != rows_pad:
        raise ValueError("shape mismatch")
    if workspace is None:
        workspace = gemm_workspace(n, t, k, y.device)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    wsp = _ptr(workspace) if workspace is not None else ctypes.c_void_p(0)
    wsb = workspace.numel() if workspace is not None else 0
    args = (_ptr(w), n, k, _ptr(qs), _ptr(ds), t, rows_pad, _ptr(y), wsp, wsb, _stream(stream))
    if bind:
        b = Bound("q8_0_gemm", args)
        b._keep = workspace
        return b
    _check("q8_0_gemm", lib().q8_0_gemm(*args))
    return None


_noalloc_devices = set()  # devices on which an eager q8_0_gemm_noalloc call has succeeded


def q8_0_gemm_noalloc(w, n: int, k: int, qs, ds, t: int, y, stream=None, bind=False):
    """q8_0_gemm whose scratch is the library's fixed device array (no allocation anywhere).

    For callers that cannot allocate device memory here; requests larger than
    q8_0_gemm_noalloc_max_bytes() raise Q8Error(Q8_ERR_TOO_BIG).  Calls that overlap
    on the GPU share that array and race.  The first call on a device looks the
    array up (a host-side CUDA call), so ``bind=True`` -- the form used to record
    launches into a CUDA graph -- is refused until one eager call has been made on
    that device."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    rows_pad = qs.shape[0]
    if w.numel() != n * (k // 32) * 34 or y.numel() < t * n or qs.shape[-1] != k or ds.shape[0] != rows_pad:
        raise ValueError("shape mismatch")
    dev = y.device.index if y.device.index is not None else torch.cuda.current_device()
    if bind and dev not in _noalloc_devices:
        raise RuntimeError("q8_0_gemm_noalloc: make one eager call on this device before binding it (its first call "
                           "looks up the scratch array's device address, which must not happen inside a stream capture)")
    out = _launch("q8_0_gemm_noalloc", (_ptr(w), n, k, _ptr(qs), _ptr(ds), t, rows_pad, _ptr(y), _stream(stream)),
                  bind)
    if not bind:
        _noalloc_devices.add(dev)
    return out


def q8_0_gemm_mma(w, n: int, k: int, qs, ds, t: int, y, stream=None, bind=False):
    """Legacy-tensor-path A/B twin of :func:`q8_0_gemm` (mma.sync.m16n8k32.s8)."""
    import torch

    _need(w, torch.uint8, "w"), _need(qs, torch.int8, "qs"), _need(ds, torch.int32, "ds"), _need(y, torch.float32, "y")
    rows_pad = qs.shape[0]
    if w.numel() != n * (k // 32) * 34 or y.numel() < t * n or qs.shape[-1] != k or ds.shape[0] != rows_pad:
        raise ValueError("shape mismatch")
    return _launch("q8_0_gemm_mma", (_ptr(w), n, k, _ptr(qs), _ptr(ds), t, rows_pad, _ptr(y), _stream(stream)), bind)


def empty_kv_cache(layers: int, n_pages: int, kv_heads: int, page_size: int, head_dim: int, int8: bool = False,
                   device="cuda") -> KvCache:
    """Allocate (with PyTorch) an uninitialised paged cache, f16 or int8 with f32 scales."""
    import torch

    shape = (layers, n_pages, kv_heads, page_size, head_dim)
    dt = torch.int8 if int8 else torch.float16
    k, v = (torch.empty(shape, dtype=dt, device=device) for _ in range(2))
    ks, vs = (torch.empty(shape[:-1], dtype=torch.float32, device=device) if int8 else None for _ in range(2))
    return KvCache(k, v, ks, vs)


def _beside(t, dtype, dev, name):
    """The device pointer of a contiguous tensor of this type on CUDA device `dev`."""
    if t.dtype is not dtype or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of {dtype} on cuda:{dev}, got {t.dtype} on {t.device}")
    return t.data_ptr()


_kv_fns = {}  # entry points of the loaded library
_workspace_sizes = {}  # of q8_tree_attention, by the sizes they depend on


def _kv_call(name, args, dev, stream, bind, keep):
    """Launch (or bind) a key/value cache call on `stream`, or on the current stream of the tensors' device."""
    from torch import _C

    if dev != _C._cuda_getDevice():
        raise ValueError(f"{name}: tensors on cuda:{dev}, which is not the current device")
    if stream is None:
        stream = _C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    args += (stream,)
    if bind:
        b = Bound(name, args)
        b._keep = keep
        return b
    fn = _kv_fns.get(name)
    if fn is None:
        fn = _kv_fns[name] = getattr(lib(), name)
    st = fn(*args)
    if st != 0:
        raise Q8Error(name, st)
    return None


def q8_kv_plan(cached, fresh, free_pages, table, page_size: int, n_pages: int, starts, slots, positions, needed,
               parents=None, masks=None, held=None, held_out=None, stream=None, bind=False):
    """The integers of one step over a paged cache, from the request lengths.

    cached, fresh int32 [batch]; free_pages int32 [n_free] ids to hand out; table int32 [batch][max_pages] (the
    entries for newly opened pages are written, -1 where the list ran out); starts int32 [batch + 1], slots and
    positions int32 [tokens], needed int32 [1] are outputs.  The list itself is left: the caller drops its first
    ``needed`` ids after the step.  ``parents`` int32 [tokens] with ``masks`` int64 [tokens] (output): draft trees.
    ``held`` int32 [batch]: pages each row has already (default ceil(cached / page_size)); ``held_out``: after the step,
    a tensor of its own.  Outputs share no memory with inputs or one another (refused)."""
    import torch

    i32, dev = torch.int32, cached.get_device()
    batch, tokens, shape = cached.numel(), slots.numel(), table.shape
    n_free = free_pages.numel() if free_pages is not None else 0
    if (len(shape) != 2 or shape[0] != batch or fresh.numel() != batch or starts.numel() != batch + 1
            or positions.numel() != tokens or needed.numel() != 1 or (parents is not None and parents.numel() != tokens)
            or (masks is not None and masks.numel() != tokens) or (held is not None and held.numel() != batch)
            or (held_out is not None and held_out.numel() != batch)):
        raise ValueError("shape mismatch")
    args = (_beside(cached, i32, dev, "cached"), _beside(fresh, i32, dev, "fresh"), batch,
            _beside(held, i32, dev, "held") if held is not None else None,
            _beside(free_pages, i32, dev, "free_pages") if n_free else None, n_free, _beside(table, i32, dev, "table"),
            shape[1], page_size, n_pages, _beside(parents, i32, dev, "parents") if parents is not None else None, tokens,
            _beside(starts, i32, dev, "starts"), _beside(slots, i32, dev, "slots"),
            _beside(positions, i32, dev, "positions"),
            _beside(masks, torch.int64, dev, "masks") if masks is not None else None,
            _beside(needed, i32, dev, "needed"), _beside(held_out, i32, dev, "held_out") if held_out is not None else None)
    return _kv_call("q8_kv_plan", args, dev, stream, bind, (cached, fresh, held, free_pages, table, parents, starts, slots,
                                                            positions, masks, needed, held_out))


def q8_kv_append(cache: KvCache, layer: int, k, v, slots, stream=None, bind=False):
    """Write k, v f32 [tokens][kv_heads * head_dim] to the cache slots of one layer (int32 [tokens], < 0: skipped)."""
    import torch

    dev, tokens = cache._dev, slots.numel()
    size = tokens * cache._kv_heads * cache._head_dim
    if k.numel() != size or v.numel() != size:
        raise ValueError("k, v: expected [tokens][kv_heads * head_dim]")
    args = (cache._ref, layer, _beside(k, torch.float32, dev, "k"), _beside(v, torch.float32, dev, "v"),
            _beside(slots, torch.int32, dev, "slots"), tokens)
    return _kv_call("q8_kv_append", args, dev, stream, bind, (cache, k, v, slots))


def q8_tree_attention_workspace_bytes(cache: KvCache, heads: int, max_fresh: int) -> int:
    return int(lib().q8_tree_attention_workspace_bytes(cache._ref, heads, max_fresh))


def q8_tree_attention_needs_workspace(cache: KvCache, heads: int, batch: int, max_fresh: int, max_len: int) -> bool:
    return bool(lib().q8_tree_attention_needs_workspace(cache._ref, heads, batch, max_fresh, max_len))


def _workspace_size(cache, heads, batch, max_fresh, max_len):
    """Bytes of the workspace that a call without one gets; remembered by what they depend on."""
    key = cache._kv_heads, cache._head_dim, heads, batch, max_fresh, max_len
    nbytes = _workspace_sizes.get(key)
    if nbytes is None:
        nbytes = 0
        if q8_tree_attention_needs_workspace(cache, heads, batch, max_fresh, max_len):
            nbytes = q8_tree_attention_workspace_bytes(cache, heads, max_fresh)
            if nbytes == 0:  # sizes or a descriptor that the call refuses: another cache with these figures may be right
                return 0
        if len(_workspace_sizes) < 1024:
            _workspace_sizes[key] = nbytes
    return nbytes


def q8_tree_attention(cache: KvCache, layer: int, q, table, cached, starts, y, qs=None, ds=None, masks=None,
                      max_fresh: int = 0, max_len: int = 0, scale: float | None = None, workspace=None, stream=None,
                      bind=False):
    """Attention of a step's fresh tokens over the paged cache.

    q f32 [tokens][heads * head_dim]; table, cached, starts as :func:`q8_kv_plan` left them; ``masks`` int64
    [tokens] of draft trees, or None for causal.  Writes ``y`` (f32, like q; None when dead) and, with ``qs``/``ds``,
    its q8_0 plane.  ``max_fresh`` (default tokens; with masks at most TREE_MAX_NODES) and ``max_len`` (default the
    table's width) bound the lengths of a sequence.  ``max_fresh`` decides how many rows a unit has: give it for a batch
    of several sequences (61 single tokens over up to 8191 keys take 219 us with the default, 76 with 1, int8).
    ``scale`` defaults to 1/sqrt(head_dim).  ``workspace``: a uint8 CUDA tensor of at least
    q8_tree_attention_workspace_bytes(...) bytes; when None, and the call needs one, it is allocated here with PyTorch."""
    import torch

    dev, dim, i32 = cache._dev, cache._head_dim, torch.int32
    size, shape, tshape = q.numel(), q.shape, table.shape
    batch = cached.numel()
    if len(shape) != 2 or shape[1] % dim or len(tshape) != 2 or tshape[0] != batch or starts.numel() != batch + 1:
        raise ValueError("q: expected [tokens][heads * head_dim]; table [batch][max_pages], starts [batch + 1]")
    tokens, heads = shape[0], shape[1] // dim
    if ((y is not None and y.numel() < size) or (qs is not None and qs.numel() < size)
            or (ds is not None and ds.numel() < size // 32) or (masks is not None and masks.numel() < tokens)):
        raise ValueError("y, qs, ds or masks: fewer rows than q")
    if not max_fresh:
        max_fresh = tokens if masks is None else min(tokens, TREE_MAX_NODES)
    max_len = max_len or tshape[1] * cache._page_size
    if workspace is None:
        nbytes = _workspace_size(cache, heads, batch, max_fresh, max_len)
        if nbytes == 0:
            pass
        elif stream is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache._k.device)
        else:  # from the pool of the stream that uses it, so that it is not handed out again too early
            with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache._k.device)
    args = (cache._ref, layer, _beside(q, torch.float32, dev, "q"), heads, dim ** -0.5 if scale is None else scale,
            _beside(table, i32, dev, "table"), tshape[1], _beside(cached, i32, dev, "cached"),
            _beside(starts, i32, dev, "starts"), batch,
            _beside(masks, torch.int64, dev, "masks") if masks is not None else None, tokens, max_fresh,
            max_len, _beside(y, torch.float32, dev, "y") if y is not None else None,
            _beside(qs, torch.int8, dev, "qs") if qs is not None else None,
            _beside(ds, i32, dev, "ds") if ds is not None else None,
            _beside(workspace, torch.uint8, dev, "workspace") if workspace is not None else None,
            workspace.numel() if workspace is not None else 0)
    return _kv_call("q8_tree_attention", args, dev, stream, bind, (cache, q, table, cached, starts, masks, y, qs, ds,
                                                                   workspace))


def q8_kv_accept(cache: KvCache, table, cached, fresh, paths, counts, lens, stream=None, bind=False):
    """Move each sequence's accepted path (paths int32 [batch][width], counts int32 [batch]) to the front of its
    fresh tokens, in every layer; lens int32 [batch] (output, not in the place of ``cached``) = cached + counts."""
    import torch

    dev, i32 = cache._dev, torch.int32
    batch, tshape, pshape = cached.numel(), table.shape, paths.shape
    if (len(tshape) != 2 or tshape[0] != batch or len(pshape) != 2 or pshape[0] != batch or fresh.numel() != batch
            or counts.numel() != batch or lens.numel() != batch):
        raise ValueError("shape mismatch")
    args = (cache._ref, _beside(table, i32, dev, "table"), tshape[1], _beside(cached, i32, dev, "cached"),
            _beside(fresh, i32, dev, "fresh"), batch, _beside(paths, i32, dev, "paths"),
            _beside(counts, i32, dev, "counts"), pshape[1], _beside(lens, i32, dev, "lens"))
    return _kv_call("q8_kv_accept", args, dev, stream, bind, (cache, table, cached, fresh, paths, counts, lens))


def _scratch(workspace, nbytes, dev, stream):
    """The caller's workspace, or one of `nbytes` from the pool of the stream that uses it; None where none is needed."""
    import torch

    if workspace is not None or not nbytes:
        return workspace
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")


def _opt(t, dtype, dev, name):
    return _beside(t, dtype, dev, name) if t is not None else None


def _scratch_args(workspace, dev):
    return (_beside(workspace, workspace.dtype, dev, "workspace"), workspace.nbytes) if workspace is not None else (None, 0)


def q8_moe_route_workspace_bytes(tokens: int, experts: int, top_k: int) -> int:
    return int(lib().q8_moe_route_workspace_bytes(tokens, experts, top_k))


def q8_moe_route(logits, ids, weights, offsets, rows, places, mode: int = ROUTE_CHOSEN, scale: float = 1.0, valid=None,
                 workspace=None, stream=None, bind=False):
    """The top_k experts of each token, their weights, and the (token, expert) pairs sorted by expert.

    logits f32 [tokens][experts]; outputs ids int32 and weights f32 [tokens][top_k], offsets int32 [experts + 1], rows
    int32 [tokens * top_k] (the pair of each sorted row), places int32 [tokens][top_k] (the sorted row of each pair).
    ``mode``: ROUTE_CHOSEN or ROUTE_ALL, what the softmax of the weights runs over.  ``valid`` int32 [1]: how many tokens
    count (default all).  ``workspace``: a uint8 CUDA tensor; allocated here with PyTorch when None and one is needed."""
    import torch

    i32, dev = torch.int32, logits.get_device()
    shape, ishape = logits.shape, ids.shape
    if len(shape) != 2 or len(ishape) != 2 or ishape[0] != shape[0]:
        raise ValueError("logits: expected [tokens][experts]; ids [tokens][top_k]")
    (tokens, experts), top_k = shape, ishape[1]
    if (weights.shape != ishape or places.shape != ishape or offsets.numel() != experts + 1
            or rows.numel() != tokens * top_k or (valid is not None and valid.numel() != 1)):
        raise ValueError("shape mismatch")
    args = (_beside(logits, torch.float32, dev, "logits"), tokens, experts, top_k, mode, scale,
            _opt(valid, i32, dev, "valid"), _beside(ids, i32, dev, "ids"), _beside(weights, torch.float32, dev, "weights"),
            _beside(offsets, i32, dev, "offsets"), _beside(rows, i32, dev, "rows"), _beside(places, i32, dev, "places"))
    workspace = _scratch(workspace, q8_moe_route_workspace_bytes(tokens, experts, top_k), dev, stream)
    return _kv_call("q8_moe_route", args + _scratch_args(workspace, dev), dev, stream, bind,
                    (logits, valid, ids, weights, offsets, rows, places, workspace))


def _experts_sizes(w, experts, n, k, qs, ds, offsets, rows, top_k, pairs):
    if k % 32 or w.numel() != experts * n * (k // 32) * 34:
        raise ValueError("w: expected experts * n rows of k/32 blocks of 34 bytes")
    shape = qs.shape
    if len(shape) != 2 or shape[1] != k or ds.shape != (shape[0], k // 32):
        raise ValueError("plane shape mismatch")
    if offsets.numel() != experts + 1 or (rows is not None and rows.numel() != pairs):
        raise ValueError("offsets: expected [experts + 1]; rows [pairs]")
    return (experts, n, k, shape[0], top_k, pairs)


def q8_0_experts_gemm_workspace_bytes(experts: int, n: int, k: int, plane_rows: int, top_k: int, pairs: int) -> int:
    return int(lib().q8_0_experts_gemm_workspace_bytes(experts, n, k, plane_rows, top_k, pairs))


def q8_0_experts_gemm(w, experts: int, n: int, k: int, qs, ds, offsets, y, rows=None, top_k: int = 1, workspace=None,
                      stream=None, bind=False):
    """y f32 [pairs][n]: each sorted row's plane row times its expert's matrix.

    w uint8 [experts][n][k/32 blocks of 34 bytes]; offsets int32 [experts + 1] and ``rows`` int32 [pairs] as
    :func:`q8_moe_route` wrote them with this ``top_k`` (row r reads plane row rows[r] // top_k), or ``rows=None``: row r
    reads plane row r.  Rows behind offsets[experts] are left.  ``workspace``: a uint8 CUDA tensor of at least
    q8_0_experts_gemm_workspace_bytes(...) bytes; allocated here with PyTorch when None and one is needed."""
    import torch

    i32, dev, pairs = torch.int32, qs.get_device(), y.shape[0]
    if y.numel() != pairs * n:
        raise ValueError("y: expected [pairs][n]")
    sizes = _experts_sizes(w, experts, n, k, qs, ds, offsets, rows, top_k, pairs)
    workspace = _scratch(workspace, q8_0_experts_gemm_workspace_bytes(*sizes), dev, stream)
    args = (_beside(w, torch.uint8, dev, "w"), experts, n, k, _beside(qs, torch.int8, dev, "qs"), _beside(ds, i32, dev, "ds"),
            sizes[3], _beside(offsets, i32, dev, "offsets"), _opt(rows, i32, dev, "rows"), top_k, pairs,
            _beside(y, torch.float32, dev, "y"))
    return _kv_call("q8_0_experts_gemm", args + _scratch_args(workspace, dev), dev, stream, bind,
                    (w, qs, ds, offsets, rows, y, workspace))


def q8_0_experts_gate_up_workspace_bytes(experts: int, nf: int, k: int, plane_rows: int, top_k: int, pairs: int) -> int:
    return int(lib().q8_0_experts_gate_up_workspace_bytes(experts, nf, k, plane_rows, top_k, pairs))


def q8_0_experts_gate_up(w_gate, w_up, experts: int, nf: int, k: int, qs, ds, offsets, qs_out, ds_out, rows=None,
                         top_k: int = 1, workspace=None, stream=None, bind=False):
    """The plane (qs_out int8 [>= pairs][nf], ds_out int32 [>= pairs][nf/32]) of silu(gate) * up of the sorted rows.

    w_gate, w_up and the other arguments as for :func:`q8_0_experts_gemm`; the plane's rows are in sorted order, ready for
    the down product with ``rows=None``.  ``pairs`` is rows' length, or the output plane's rows without ``rows``."""
    import torch

    i32, dev = torch.int32, qs.get_device()
    oshape = qs_out.shape
    pairs = rows.numel() if rows is not None else oshape[0]
    if len(oshape) != 2 or oshape[1] != nf or oshape[0] < pairs or ds_out.shape != (oshape[0], nf // 32):
        raise ValueError("output plane shape mismatch")
    sizes = _experts_sizes(w_gate, experts, nf, k, qs, ds, offsets, rows, top_k, pairs)
    if w_up.numel() != w_gate.numel():
        raise ValueError("w_up: expected the size of w_gate")
    workspace = _scratch(workspace, q8_0_experts_gate_up_workspace_bytes(*sizes), dev, stream)
    args = (_beside(w_gate, torch.uint8, dev, "w_gate"), _beside(w_up, torch.uint8, dev, "w_up"), experts, nf, k,
            _beside(qs, torch.int8, dev, "qs"), _beside(ds, i32, dev, "ds"), sizes[3], _beside(offsets, i32, dev, "offsets"),
            _opt(rows, i32, dev, "rows"), top_k, pairs, _beside(qs_out, torch.int8, dev, "qs_out"),
            _beside(ds_out, i32, dev, "ds_out"))
    return _kv_call("q8_0_experts_gate_up", args + _scratch_args(workspace, dev), dev, stream, bind,
                    (w_gate, w_up, qs, ds, offsets, rows, qs_out, ds_out, workspace))


def rmsnorm_residual_quant(x, h, b=None, expert_rows=None, places=None, weights=None, w_post=None, eps_post: float = 0.0,
                           gate=None, residual_scale: float = 1.0, w=None, eps: float = 0.0, y=None, qs=None, ds=None,
                           stream=None, bind=False):
    """h = residual_scale * x + gate * norm(b + sum_j weights[:, j] * expert_rows[places[:, j]]), then y = rmsnorm(h) * w
    and its plane, in one pass.

    x, b, h (``x`` itself allowed; None when dead) and y f32 [rows][d]; expert_rows f32 [pairs][d], places int32 and
    weights f32 [rows][top_k] (q8_moe_route's; -1 adds nothing); w_post (None: no norm behind the block) and w f32 [d]; gate
    f32 [1][d] or [rows][d].  ``y`` and the plane (``qs``/``ds``, any padded rows) are optional and need ``w``."""
    import torch

    f32, i32, dev = torch.float32, torch.int32, x.get_device()
    rows, d = x.shape
    top_k = 0
    if expert_rows is not None:
        if places is None or weights is None or len(places.shape) != 2 or weights.shape != places.shape:
            raise ValueError("places, weights: expected [rows][top_k] with expert_rows")
        top_k = places.shape[1]
        if places.shape[0] != rows or top_k < 1 or len(expert_rows.shape) != 2 or expert_rows.shape[1] != d:
            raise ValueError("expert_rows: expected [pairs][d]; places [rows][top_k]")
    elif places is not None or weights is not None:
        raise ValueError("places and weights with expert_rows, and only then")
    for t, name in ((b, "b"), (h, "h"), (y, "y")):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name}: expected the shape of x")
    if (w is not None and w.numel() != d) or (w_post is not None and w_post.numel() != d):
        raise ValueError("w, w_post: expected [d]")
    if gate is not None and (gate.numel() % d or gate.numel() // d not in (1, rows)):
        raise ValueError("gate: expected [1][d] or [rows][d]")
    rows_pad = qs.shape[0] if qs is not None else 0
    if (qs is None) != (ds is None) or (qs is not None and (qs.shape != (rows_pad, d) or ds.shape != (rows_pad, d // 32))):
        raise ValueError("plane shape mismatch")
    args = (_beside(x, f32, dev, "x"), residual_scale, _opt(b, f32, dev, "b"), _opt(expert_rows, f32, dev, "expert_rows"),
            expert_rows.shape[0] if top_k else 0, _opt(places, i32, dev, "places"), _opt(weights, f32, dev, "weights"), top_k,
            _opt(w_post, f32, dev, "w_post"), eps_post, _opt(gate, f32, dev, "gate"), gate.numel() // d if gate is not None else 0,
            _opt(w, f32, dev, "w"), eps, _opt(h, f32, dev, "h"), _opt(y, f32, dev, "y"), rows, d,
            _opt(qs, torch.int8, dev, "qs"), _opt(ds, i32, dev, "ds"), rows_pad)
    return _kv_call("rmsnorm_residual_quant", args, dev, stream, bind, (x, b, expert_rows, places, weights, w_post, gate, w, h, y,
                                                                        qs, ds))


def empty_plane(rows_pad: int, k: int, device="cuda"):
    """Allocate (with PyTorch) an uninitialised plane: (qs int8, ds int32)."""
    import torch

    return (torch.empty((rows_pad, k), dtype=torch.int8, device=device),
            torch.empty((rows_pad, k // 32), dtype=torch.int32, device=device))
