"""QK-Norm on MI355X (gfx950): Python binding of the C-ABI library.

This module only marshals arguments: torch tensors supply device pointers and
the current HIP stream, and every step of the computation runs in the HIP
kernels of ``libqknorm.so``.  There is no CPU fallback -- if the library is
not built, or a tensor is not on the GPU, the call raises.

The entry points keep the C names and semantics (``include/qknorm.h``).  The norms:

    qknorm_per_head(qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps)
    qknorm_layerwise(qkv, wq, wk, gamma_q, gamma_k, eps, nshards)
    qknorm_partial_sumsq(qkv, wq, wk, nshards, part_q, part_k)
    qknorm_apply_scalar(qkv, wq, wk, part_q, part_k, norm_wq, norm_wk, gamma_q, gamma_k, eps)

``qkv`` is float32, bfloat16 or float16 with gamma of the same dtype, or
float8_e4m3fn with bfloat16 gamma.  It is a [T, ...] tensor whose rows are
contiguous within themselves
(``stride(-1) == 1`` and each row packed); its row pitch is ``stride(0)``.
They normalise in place.  Beside them the QKV projection with the norm in its
epilogue (``qknorm_qkv_proj_per_head`` and its workspace forms), and an
attention block's low-bit path:

    qknorm_quant_rows(x, q, scale)
    qknorm_qkv_proj_quant(x, x_scale, w, w_scale, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps)
    qknorm_kv_append(qkv, hq, hkv, head_dim, cache, slots)
    qknorm_kv_gather(cache, slots, k, v, hkv, head_dim)
    qknorm_kv_attention(qkv, cache, page_table, seq_lens, out, hq, hkv, head_dim)

All calls are enqueued on ``stream`` (default: torch's current stream).
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqknorm.so")

QKNORM_F32 = 0
QKNORM_BF16 = 1
QKNORM_F16 = 2
QKNORM_FP8_E4M3 = 3
QKNORM_OK = 0
QKNORM_E_NULLPTR = -1
QKNORM_E_SHAPE = -2
QKNORM_E_ALIGN = -3
QKNORM_E_DTYPE = -4
QKNORM_E_UNSUPPORTED = -5
QKNORM_E_EPS = -6
QKNORM_E_HIP = -7

QKNORM_PROJ_PLAIN = 1
QKNORM_KV_PAGE = 64    # tokens a page of the 4-bit cache holds

EXPORTED = ("qknorm_per_head", "qknorm_layerwise", "qknorm_partial_sumsq",
            "qknorm_apply_scalar", "qknorm_qkv_proj_per_head", "qknorm_qkv_proj_workspace_bytes",
            "qknorm_qkv_proj_per_head_ws", "qknorm_qkv_proj_per_head_noalloc", "qknorm_quant_rows",
            "qknorm_qkv_proj_quant", "qknorm_qkv_proj_quant_workspace_bytes", "qknorm_kv_page_bytes",
            "qknorm_kv_append", "qknorm_kv_gather", "qknorm_kv_attention",
            "qknorm_kv_attention_workspace_bytes", "qknorm_strerror", "qknorm_abi_version")

_lib = None


class QKNormError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (code {code})")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"QK-Norm HIP library not built: {path} is missing "
                           "(run `python -m qk_norm_amd.build` or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    lib.qknorm_per_head.argtypes = [P, I64, I64, I32, I32, I32, P, P, F, I32, P]
    lib.qknorm_layerwise.argtypes = [P, I64, I64, I64, I64, P, P, F, I32, I32, P]
    lib.qknorm_partial_sumsq.argtypes = [P, I64, I64, I64, I64, I32, P, P, I32, P]
    lib.qknorm_apply_scalar.argtypes = [P, I64, I64, I64, I64, P, P, I32, I64, I64, P, P, F, I32, P]
    lib.qknorm_qkv_proj_per_head.argtypes = [P, I64, P, I64, P, I64, I64, I64, I32, I32, I32, P, P,
                                             F, I32, I32, P]
    lib.qknorm_qkv_proj_workspace_bytes.argtypes = [I64, I32, I32, I32]
    lib.qknorm_qkv_proj_workspace_bytes.restype = I64
    lib.qknorm_qkv_proj_per_head_ws.argtypes = [P, I64, P, I64, P, I64, I64, I64, I32, I32, I32, P, P,
                                                F, I32, I32, P, I64, P]
    lib.qknorm_qkv_proj_per_head_noalloc.argtypes = lib.qknorm_qkv_proj_per_head.argtypes
    lib.qknorm_quant_rows.argtypes = [P, I64, P, I64, P, I64, I64, I32, P]
    lib.qknorm_qkv_proj_quant.argtypes = [P, I64, P, P, I64, P, P, I64, I64, I64, I32, I32, I32, P, P, F, I32, I32,
                                         P, I64, P]
    lib.qknorm_kv_append.argtypes = [P, I64, I64, I32, I32, I32, P, I64, I64, P, I32, P]
    lib.qknorm_kv_gather.argtypes = [P, I64, I64, P, I64, I32, I32, P, I64, P, I64, I32, P]
    lib.qknorm_kv_attention.argtypes = [P, I64, I64, P, I64, I64, P, I64, I64, P, P, I64, P, I64, P, I32, I32, I32,
                                         F, I32, I32, P, I64, P]
    for name, args in (("qknorm_qkv_proj_quant_workspace_bytes", [I64, I32, I32, I32]),
                       ("qknorm_kv_page_bytes", [I32, I32]),
                       ("qknorm_kv_attention_workspace_bytes", [I64, I64, I64, I32, I32, I32])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = I64
    for name in ("qknorm_per_head", "qknorm_layerwise", "qknorm_partial_sumsq",
                 "qknorm_apply_scalar", "qknorm_qkv_proj_per_head", "qknorm_qkv_proj_per_head_ws",
                 "qknorm_qkv_proj_per_head_noalloc", "qknorm_quant_rows", "qknorm_qkv_proj_quant",
                 "qknorm_kv_append", "qknorm_kv_gather", "qknorm_kv_attention", "qknorm_abi_version"):
        getattr(lib, name).restype = I32
    lib.qknorm_strerror.argtypes = [ctypes.c_int]
    lib.qknorm_strerror.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


_calls_mod = None       # the CPython call module (or its ctypes stand-in)


class _CtypesCalls:
    """The call module's functions through ctypes, for a tree where the module
    is not built (the same library calls, only slower to make)."""

    def __init__(self, lib):
        self.per_head = lib.qknorm_per_head
        self.layerwise = lib.qknorm_layerwise
        self.partial_sumsq = lib.qknorm_partial_sumsq
        self.apply_scalar = lib.qknorm_apply_scalar
        self.qkv_proj_per_head = lib.qknorm_qkv_proj_per_head
        self.qkv_proj_per_head_ws = lib.qknorm_qkv_proj_per_head_ws
        self.qkv_proj_per_head_noalloc = lib.qknorm_qkv_proj_per_head_noalloc
        self.quant_rows = lib.qknorm_quant_rows
        self.qkv_proj_quant = lib.qknorm_qkv_proj_quant
        self.kv_append = lib.qknorm_kv_append
        self.kv_gather = lib.qknorm_kv_gather
        self.kv_attention = lib.qknorm_kv_attention

    @staticmethod
    def per_head_t(*_):
        return None

    layerwise_t = quant_rows_t = qkv_proj_quant_t = kv_append_t = kv_gather_t = kv_attention_t = per_head_t


def _calls():
    """The functions that call the C ABI: `_qknorm_fast` (qk_norm_amd/csrc/pyfast.cpp),
    which converts the Python ints and floats itself and, for the common case of
    contiguous GPU tensors, reads the tensors itself too; or ctypes."""
    global _calls_mod
    if _calls_mod is None:
        lib = load()
        try:
            from . import _qknorm_fast as mod
        except ImportError:
            mod = _CtypesCalls(lib)
        else:
            import torch
            if _CODES is None:
                _torch_tables()
            mod.setup(_raw_stream, torch.Tensor)
        _calls_mod = mod
    return _calls_mod


def strerror(code: int) -> str:
    return load().qknorm_strerror(int(code)).decode()


def abi_version() -> int:
    return int(load().qknorm_abi_version())


# ----------------------------------------------------------------- marshal --

# Everything below runs on every call, so it sticks to cheap tensor
# attributes (shape, stride, dtype, device index) and the raw stream handle.

_CODES = None           # torch dtype -> (dtype code, gamma dtype)
_raw_stream = None      # device index -> current hipStream_t as an int


def _torch_tables():
    global _CODES, _raw_stream
    import torch
    _CODES = {torch.float32: (QKNORM_F32, torch.float32),
              torch.bfloat16: (QKNORM_BF16, torch.bfloat16),
              torch.float16: (QKNORM_F16, torch.float16),
              torch.float8_e4m3fn: (QKNORM_FP8_E4M3, torch.bfloat16)}
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = raw if raw is not None else (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _dtype_code(t) -> int:
    if _CODES is None:
        _torch_tables()
    try:
        return _CODES[t.dtype][0]
    except KeyError:
        raise ValueError("QK-Norm supports float32, bfloat16, float16 and float8_e4m3fn tensors, "
                         f"not {t.dtype}") from None


def _rows(qkv):
    """(T, ld, device index) of a [T, ...] GPU tensor whose rows are packed."""
    if not qkv.is_cuda:
        raise ValueError("qkv must be a GPU tensor (the library has no CPU path)")
    if qkv.is_contiguous() and qkv.dim() >= 2:
        T = qkv.shape[0]
        if T > 0:                # rows back to back: the pitch is the row's size
            return T, qkv.numel() // T, qkv.get_device()
    shape, stride = qkv.shape, qkv.stride()
    if len(shape) < 2:
        raise ValueError("qkv must have a leading token dimension and at least one more")
    T = shape[0]
    row = 1                      # elements per row, and the check that they are packed
    for n, st in zip(reversed(shape[1:]), reversed(stride[1:])):
        if T > 0 and n != 1 and st != row:
            raise ValueError("each qkv row must be contiguous")
        row *= n
    ld = stride[0] if T > 1 else max(stride[0], row)
    return T, ld, qkv.get_device()


def _ptr(t, dev):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    if t.get_device() != dev:
        raise ValueError("all tensors must be on the same GPU")
    return t.data_ptr()


def _gamma(g, qkv, dev):
    if g is None:
        return None
    if _CODES is None:
        _torch_tables()
    want = _CODES[qkv.dtype][1] if qkv.dtype in _CODES else qkv.dtype
    if g.dtype != want:
        raise ValueError(f"gamma must be {want} for {qkv.dtype} activations")
    if not g.is_contiguous():
        raise ValueError("gamma must be contiguous")
    return _ptr(g, dev)


def _stream(stream, dev):
    if stream is None:
        if _raw_stream is None:
            _torch_tables()
        return _raw_stream(dev)
    return getattr(stream, "cuda_stream", stream)


def _raise(rc: int, what: str):
    if rc == QKNORM_OK:
        return
    if rc == QKNORM_E_HIP:
        raise QKNormError(rc, what)
    raise ValueError(f"{what}: {strerror(rc)} (code {rc})")


# -------------------------------------------------------------- entry points --

def qknorm_per_head(qkv, hq: int, hkv: int, head_dim: int, gamma_q, gamma_k=None,
                    eps: float = 1e-6, stream=None) -> None:
    """Per-head RMSNorm of the hq Q heads and hkv K heads of each row, in place."""
    c = _calls_mod or _calls()
    rc = c.per_head_t(qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, stream)
    if rc is None:               # not the common case: the full checks, in Python
        T, ld, dev = _rows(qkv)
        rc = c.per_head(qkv.data_ptr(), T, ld, hq, hkv, head_dim, _gamma(gamma_q, qkv, dev),
                        _gamma(gamma_k, qkv, dev), eps, _dtype_code(qkv), _stream(stream, dev))
    if rc:
        _raise(rc, "qknorm_per_head")


def qknorm_layerwise(qkv, wq: int, wk: int, gamma_q, gamma_k=None, eps: float = 1e-6,
                     nshards: int = 1, stream=None) -> None:
    """Layerwise RMSNorm over the whole Q and K widths via nshards partials, in place."""
    c = _calls_mod or _calls()
    rc = c.layerwise_t(qkv, wq, wk, gamma_q, gamma_k, eps, nshards, stream)
    if rc is None:               # not the common case: the full checks, in Python
        T, ld, dev = _rows(qkv)
        rc = c.layerwise(qkv.data_ptr(), T, ld, wq, wk, _gamma(gamma_q, qkv, dev),
                         _gamma(gamma_k, qkv, dev), eps, nshards, _dtype_code(qkv), _stream(stream, dev))
    if rc:
        _raise(rc, "qknorm_layerwise")


def _partials(p, dev):
    import torch
    if p is None:
        return None
    if p.dtype != torch.float32 or not p.is_contiguous():
        raise ValueError("partials must be contiguous float32 [nshards, T]")
    return _ptr(p, dev)


def qknorm_partial_sumsq(qkv, wq: int, wk: int, nshards: int, part_q, part_k,
                         stream=None) -> None:
    """Shard partial sums of squares into part_q / part_k, float32 [nshards, T]."""
    T, ld, dev = _rows(qkv)
    rc = _calls().partial_sumsq(qkv.data_ptr(), T, ld, wq, wk, nshards,
                                               _partials(part_q, dev), _partials(part_k, dev),
                                               _dtype_code(qkv), _stream(stream, dev))
    _raise(rc, "qknorm_partial_sumsq")


def qknorm_apply_scalar(qkv, wq: int, wk: int, part_q, part_k, norm_wq: int, norm_wk: int,
                        gamma_q, gamma_k=None, eps: float = 1e-6, nparts: int | None = None,
                        stream=None) -> None:
    """Combine nparts partials per token and apply, in place."""
    T, ld, dev = _rows(qkv)
    if nparts is None:
        ref = part_q if part_q is not None else part_k
        nparts = ref.shape[0] if ref is not None else 1
    rc = _calls().apply_scalar(qkv.data_ptr(), T, ld, wq, wk,
                                              _partials(part_q, dev), _partials(part_k, dev),
                                              nparts, norm_wq, norm_wk, _gamma(gamma_q, qkv, dev),
                                              _gamma(gamma_k, qkv, dev), eps, _dtype_code(qkv),
                                              _stream(stream, dev))
    _raise(rc, "qknorm_apply_scalar")


def _matrix(t, dev, what):
    """(pointer, row pitch) of a 2-d GPU tensor with contiguous rows."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a 2-d tensor with contiguous rows")
    return _ptr(t, dev), t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _proj_args(x, w, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, plain):
    """The C ABI's arguments of a projection call up to `dtype` (the stream is
    added by the caller)."""
    if not qkv.is_cuda:
        raise ValueError("qkv must be a GPU tensor (the library has no CPU path)")
    dev = qkv.get_device()
    xp, ldx = _matrix(x, dev, "x")
    wp, ldw = _matrix(w, dev, "w")
    op, ld = _matrix(qkv, dev, "qkv")
    if x.dtype != qkv.dtype or w.dtype != qkv.dtype:
        raise ValueError("x, w and qkv must share the dtype")
    if x.shape[0] != qkv.shape[0] or x.shape[1] != w.shape[1]:
        raise ValueError("x [T, hidden], w [N, hidden] and qkv [T, >= N] do not match")
    return dev, (xp, ldx, wp, ldw, op, ld, x.shape[0], x.shape[1], hq, hkv, head_dim,
                 None if plain else _gamma(gamma_q, qkv, dev), None if plain else _gamma(gamma_k, qkv, dev),
                 eps, QKNORM_PROJ_PLAIN if plain else 0, _dtype_code(qkv))


def qknorm_qkv_proj_per_head(x, w, qkv, hq: int, hkv: int, head_dim: int, gamma_q=None,
                             gamma_k=None, eps: float = 1e-6, plain: bool = False,
                             stream=None) -> None:
    """qkv[:, :N] = x @ w.T with each Q and K head RMS-normalised in the epilogue.

    x [T, hidden], w [N, hidden] (N = (hq + 2*hkv) * head_dim) and qkv [T, >= N],
    all bfloat16 or all float16 (gamma too) on one GPU; plain=True gives the
    projection alone.
    """
    dev, args = _proj_args(x, w, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, plain)
    rc = _calls().qkv_proj_per_head(*args, _stream(stream, dev))
    _raise(rc, "qknorm_qkv_proj_per_head")


def qknorm_qkv_proj_workspace_bytes(T: int, hq: int, hkv: int, head_dim: int) -> int:
    """Bytes of workspace qknorm_qkv_proj_per_head_ws needs (0: none)."""
    n = int(load().qknorm_qkv_proj_workspace_bytes(int(T), int(hq), int(hkv), int(head_dim)))
    if n < 0:
        _raise(n, "qknorm_qkv_proj_workspace_bytes")
    return n


def qknorm_qkv_proj_per_head_ws(x, w, qkv, hq: int, hkv: int, head_dim: int, gamma_q=None,
                                gamma_k=None, eps: float = 1e-6, plain: bool = False,
                                workspace=None, stream=None) -> None:
    """qknorm_qkv_proj_per_head with a workspace: a GPU tensor of at least
    qknorm_qkv_proj_workspace_bytes(T, hq, hkv, head_dim) bytes, contiguous, on
    qkv's device, that no other call uses meanwhile (None where that is 0)."""
    dev, args = _proj_args(x, w, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, plain)
    if workspace is None:
        wsp, nbytes = None, 0
    else:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        wsp, nbytes = _ptr(workspace, dev), workspace.numel() * workspace.element_size()
    rc = _calls().qkv_proj_per_head_ws(*args, wsp, nbytes, _stream(stream, dev))
    _raise(rc, "qknorm_qkv_proj_per_head_ws")


def qknorm_qkv_proj_per_head_noalloc(x, w, qkv, hq: int, hkv: int, head_dim: int, gamma_q=None,
                                     gamma_k=None, eps: float = 1e-6, plain: bool = False,
                                     stream=None) -> None:
    """qknorm_qkv_proj_per_head_ws with the library's own per-GPU scratch in
    place of a workspace (nothing allocated; calls that overlap on one GPU race)."""
    dev, args = _proj_args(x, w, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, plain)
    rc = _calls().qkv_proj_per_head_noalloc(*args, _stream(stream, dev))
    _raise(rc, "qknorm_qkv_proj_per_head_noalloc")


# ------------------------------------------------- 8-bit and 4-bit operators --

def _on(dev, fn, *args):
    """The call with the tensors' device current (kernels are launched there)."""
    import torch
    if torch._C._cuda_getDevice() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _packed_rows(t, what, dev=None):
    """(pointer, T, row width, row pitch) of a [T, ...] GPU tensor with packed rows."""
    try:
        T, ld, d = _rows(t)
    except ValueError as e:
        raise ValueError(str(e).replace("qkv", what)) from None
    if dev is not None and d != dev:
        raise ValueError("all tensors must be on the same GPU")
    width = 1
    for n in t.shape[1:]:
        width *= n
    return t.data_ptr(), T, width, ld


def _vector(t, dev, dtype, n, what):
    """Pointer of a contiguous tensor of n values of dtype."""
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} values")
    return _ptr(t, dev)


def _need_gpu(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor (the library has no CPU path)")
    return t.get_device()


def qknorm_quant_rows(x, q, scale, stream=None) -> None:
    """Rows of x to 8-bit integers, one scale a row:
    scale[t] = max|x[t]| / 127, q[t, j] = round(127 * x[t, j] / max|x[t]|), halfway to even.

    x [T, n] bfloat16 or float16, q [T, n] int8, scale [T] float32; n a multiple of 16.  For a
    projection weight [N, hidden] this is one scale per output channel.
    """
    c = _calls_mod or _calls()
    rc = c.quant_rows_t(x, q, scale, stream)
    if rc is not None:           # the common case, read in C++
        if rc:
            _raise(rc, "qknorm_quant_rows")
        return
    import torch
    dev = _need_gpu(x, "x")
    xp, ldx = _matrix(x, dev, "x")
    qp, ldq = _matrix(q, dev, "q")
    if q.dtype != torch.int8 or q.shape != x.shape:
        raise ValueError("q must be an int8 tensor of x's shape")
    sp = _vector(scale, dev, torch.float32, x.shape[0], "scale")
    rc = _on(dev, c.quant_rows, xp, ldx, qp, ldq, sp, x.shape[0], x.shape[1], _dtype_code(x),
             _stream(stream, dev))
    _raise(rc, "qknorm_quant_rows")


def qknorm_qkv_proj_quant_workspace_bytes(T: int, hq: int, hkv: int, head_dim: int) -> int:
    """Bytes of workspace with which qknorm_qkv_proj_quant takes its form for few tokens (0: none)."""
    n = int(load().qknorm_qkv_proj_quant_workspace_bytes(int(T), int(hq), int(hkv), int(head_dim)))
    if n < 0:
        _raise(n, "qknorm_qkv_proj_quant_workspace_bytes")
    return n


def _workspace(workspace, dev):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    nbytes = workspace.numel() * workspace.element_size()
    return (_ptr(workspace, dev), nbytes) if nbytes else (None, 0)


def qknorm_qkv_proj_quant(x, x_scale, w, w_scale, qkv, hq: int, hkv: int, head_dim: int, gamma_q=None,
                         gamma_k=None, eps: float = 1e-6, plain: bool = False, workspace=None,
                         stream=None) -> None:
    """qkv[:, :N] = (x @ w.T) * x_scale[:, None] * w_scale, each Q and K head RMS-normalised in the epilogue.

    x [T, hidden] and w [N, hidden] int8 (N = (hq + 2*hkv) * head_dim), x_scale [T] and w_scale
    [N] float32, as qknorm_quant_rows makes them; qkv [T, >= N] and gamma bfloat16 or float16.
    The integer product is exact.  A workspace of qknorm_qkv_proj_quant_workspace_bytes(T, ...)
    bytes (contiguous, of no other call meanwhile) speeds up 1 to 64 tokens; None is allowed.
    """
    c = _calls_mod or _calls()
    rc = c.qkv_proj_quant_t(x, x_scale, w, w_scale, qkv, hq, hkv, head_dim, gamma_q, gamma_k, eps, plain,
                            workspace, stream)
    if rc is not None:           # the common case, read in C++
        if rc:
            _raise(rc, "qknorm_qkv_proj_quant")
        return
    import torch
    dev = _need_gpu(qkv, "qkv")
    xp, ldx = _matrix(x, dev, "x")
    wp, ldw = _matrix(w, dev, "w")
    op, ld = _matrix(qkv, dev, "qkv")
    if x.dtype != torch.int8 or w.dtype != torch.int8:
        raise ValueError("x and w must be int8")
    if (x.shape[0] != qkv.shape[0] or x.shape[1] != w.shape[1] or w.shape[0] != (hq + 2 * hkv) * head_dim
            or qkv.shape[1] < w.shape[0]):
        raise ValueError("x [T, hidden], w [N, hidden] and qkv [T, >= N] do not match")
    for gamma in () if plain else (gamma_q, gamma_k):
        if gamma is not None and gamma.numel() != head_dim:
            raise ValueError("gamma must have head_dim values")
    xs = _vector(x_scale, dev, torch.float32, x.shape[0], "x_scale")
    ws = _vector(w_scale, dev, torch.float32, w.shape[0], "w_scale")
    wsp, nbytes = _workspace(workspace, dev)
    rc = _on(dev, c.qkv_proj_quant, xp, ldx, xs, wp, ldw, ws, op, ld, x.shape[0], x.shape[1], hq, hkv, head_dim,
             None if plain else _gamma(gamma_q, qkv, dev), None if plain else _gamma(gamma_k, qkv, dev), eps,
             QKNORM_PROJ_PLAIN if plain else 0, _dtype_code(qkv), wsp, nbytes, _stream(stream, dev))
    _raise(rc, "qknorm_qkv_proj_quant")


def qknorm_kv_page_bytes(hkv: int, head_dim: int) -> int:
    """Bytes of one page (64 tokens' K and V of all hkv heads) of the 4-bit cache."""
    n = int(load().qknorm_kv_page_bytes(int(hkv), int(head_dim)))
    if n < 0:
        _raise(n, "qknorm_kv_page_bytes")
    return n


def _cache(cache, dev, hkv, head_dim):
    """(pointer, pages, bytes from page to page) of a uint8 [pages, ...] cache tensor."""
    import torch
    if cache.dtype != torch.uint8:
        raise ValueError("cache must be a uint8 tensor")
    p, pages, width, stride = _packed_rows(cache, "cache", dev)
    if width != hkv * (64 * head_dim + 256):
        raise ValueError(f"a page of cache must be {hkv * (64 * head_dim + 256)} bytes, not {width}")
    return p, pages, stride


def _slots(slots, dev, T):
    import torch
    return _vector(slots, dev, torch.int64, T, "slots")


def qknorm_kv_append(qkv, hq: int, hkv: int, head_dim: int, cache, slots, stream=None) -> None:
    """Store K and V of fused rows in the paged 4-bit cache.

    qkv [T, >= (hq + 2*hkv) * head_dim] bfloat16 or float16; cache uint8 [pages, hkv, 64*head_dim
    + 256]; slots [T] int64, page * 64 + place, each named once (a row whose slot is negative or past
    the last page is skipped).
    """
    c = _calls_mod or _calls()
    rc = c.kv_append_t(qkv, hq, hkv, head_dim, cache, slots, stream)
    if rc is not None:           # the common case, read in C++
        if rc:
            _raise(rc, "qknorm_kv_append")
        return
    dev = _need_gpu(qkv, "qkv")
    qp, T, width, ld = _packed_rows(qkv, "qkv")
    if width < (hq + 2 * hkv) * head_dim:
        raise ValueError("qkv must be [T, >= (hq + 2 * hkv) * head_dim]")
    cp, pages, stride = _cache(cache, dev, hkv, head_dim)
    rc = _on(dev, c.kv_append, qp, T, ld, hq, hkv, head_dim, cp, pages, stride, _slots(slots, dev, T),
             _dtype_code(qkv), _stream(stream, dev))
    _raise(rc, "qknorm_kv_append")


def qknorm_kv_gather(cache, slots, k, v, hkv: int, head_dim: int, stream=None) -> None:
    """The K and V values held at slots [T], into k and v [T, hkv, head_dim] (float32, bfloat16 or
    float16); rows whose slot names no place are left as they are."""
    c = _calls_mod or _calls()
    rc = c.kv_gather_t(cache, slots, k, v, hkv, head_dim, stream)
    if rc is not None:           # the common case, read in C++
        if rc:
            _raise(rc, "qknorm_kv_gather")
        return
    dev = _need_gpu(cache, "cache")
    cp, pages, stride = _cache(cache, dev, hkv, head_dim)
    kp, T, wk, ldk = _packed_rows(k, "k", dev)
    vp, Tv, wv, ldv = _packed_rows(v, "v", dev)
    if Tv != T or k.dtype != v.dtype or wk != hkv * head_dim or wv != wk:
        raise ValueError("k and v must be [T, hkv, head_dim] of one dtype")
    rc = _on(dev, c.kv_gather, cp, pages, stride, _slots(slots, dev, T), T, hkv, head_dim, kp, ldk, vp, ldv,
             _dtype_code(k), _stream(stream, dev))
    _raise(rc, "qknorm_kv_gather")


def qknorm_kv_attention_workspace_bytes(T: int, B: int, max_pages: int, hq: int, hkv: int, head_dim: int) -> int:
    """Bytes of workspace that qknorm_kv_attention needs for T rows of B sequences of up to max_pages pages."""
    n = int(load().qknorm_kv_attention_workspace_bytes(int(T), int(B), int(max_pages), int(hq), int(hkv), int(head_dim)))
    if n < 0:
        _raise(n, "qknorm_kv_attention_workspace_bytes")
    return n


def qknorm_kv_attention(qkv, cache, page_table, seq_lens, out, hq: int, hkv: int, head_dim: int,
                         scale: float | None = None, q_starts=None, window: int = 0, lse=None, workspace=None,
                         stream=None) -> None:
    """Causal attention of the rows' Q heads over the paged 4-bit cache.

    qkv [T, >= hq * head_dim] bfloat16 or float16 (Q first); out [T, hq * head_dim] or [T, hq,
    head_dim] of its dtype; cache as for qknorm_kv_append; page_table [B, max_pages] and seq_lens
    [B] int32: sequence b's tokens are the first seq_lens[b] of its pages.  q_starts [B + 1] int32:
    its rows are q_starts[b] .. q_starts[b+1] - 1, the last tokens of the cache (which holds
    them already); None: row b alone.  A token sees itself and what is before it, with window > 0 the
    last `window` tokens of that; a row that sees nothing gives zeros (lse minus infinity), rows
    of no sequence are left as they are.  scale defaults to head_dim ** -0.5; lse [T, hq] float32
    receives the natural log of each row's sum of exponentials.  workspace: a contiguous tensor of at
    least qknorm_kv_attention_workspace_bytes(T, B, max_pages, hq, hkv, head_dim) bytes that no other
    call uses meanwhile.
    """
    c = _calls_mod or _calls()
    rc = c.kv_attention_t(qkv, cache, page_table, seq_lens, out, hq, hkv, head_dim,
                          head_dim ** -0.5 if scale is None else scale, q_starts, window, lse, workspace, stream)
    if rc is not None:           # the common case, read in C++
        if rc:
            _raise(rc, "qknorm_kv_attention")
        return
    import torch
    dev = _need_gpu(qkv, "qkv")
    qp, T, width, ld = _packed_rows(qkv, "qkv")
    cp, pages, stride = _cache(cache, dev, hkv, head_dim)
    op, To, wo, ldo = _packed_rows(out, "out", dev)
    if To != T or out.dtype != qkv.dtype or wo < hq * head_dim or width < hq * head_dim:
        raise ValueError("out and qkv must be [T, >= hq * head_dim] of one dtype")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be an int32 [B, max_pages] tensor with contiguous rows")
    B, max_pages = page_table.shape
    ldt = max(page_table.stride(0), max_pages) if B <= 1 else page_table.stride(0)
    lens = _vector(seq_lens, dev, torch.int32, B, "seq_lens")
    starts = None if q_starts is None else _vector(q_starts, dev, torch.int32, B + 1, "q_starts")
    lp = None if lse is None else _vector(lse, dev, torch.float32, T * hq, "lse")
    wsp, nbytes = _workspace(workspace, dev)
    rc = _on(dev, c.kv_attention, qp, T, ld, cp, pages, stride, _ptr(page_table, dev), ldt, max_pages, lens, starts,
             B, op, ldo, lp, hq, hkv, head_dim, head_dim ** -0.5 if scale is None else scale, window, _dtype_code(qkv),
             wsp, nbytes, _stream(stream, dev))
    _raise(rc, "qknorm_kv_attention")


__all__ = ["qknorm_quant_rows", "qknorm_qkv_proj_quant", "qknorm_qkv_proj_quant_workspace_bytes",
           "qknorm_kv_page_bytes", "qknorm_kv_append", "qknorm_kv_gather", "qknorm_kv_attention",
           "qknorm_kv_attention_workspace_bytes", "QKNORM_KV_PAGE", "qknorm_per_head", "qknorm_qkv_proj_per_head", "qknorm_qkv_proj_per_head_ws",
           "qknorm_qkv_proj_workspace_bytes", "qknorm_qkv_proj_per_head_noalloc", "qknorm_layerwise", "qknorm_partial_sumsq", "qknorm_apply_scalar",
           "strerror", "abi_version", "load", "QKNormError", "QKNORM_F32", "QKNORM_BF16", "QKNORM_F16",
           "QKNORM_FP8_E4M3"]
