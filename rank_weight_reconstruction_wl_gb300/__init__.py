"""Weightless linear projections on GB300: thin Python binding of libwl.so.

Every function here marshals torch CUDA tensors into the C ABI declared in
``include/wl.h`` and calls it; all arithmetic runs in the library's CUDA
kernels.  There is no Python or CPU fallback: if ``libwl.so`` is missing or a
call fails, an exception is raised.

The weightless projection ("In-kernel reconstruction", formula section):

    y[t,o] = s[o] * sum_i W0[o,i] x[t,i] + sum_k U[o,k] * sum_i V[i,k] x[t,i]

Theta arguments (``q``, ``gate`` ...) are any object with ``W0, s, U, V``
attributes, or a ``(W0, s, U, V)`` tuple.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

__all__ = [
    "WLError", "lib", "library_path", "wl_linear", "wl_qkv_fused", "wl_mlp_workspace_bytes",
    "wl_mlp_geglu_fused", "wl_mlp_geglu_fused_noalloc", "wl_materialize", "wl_decompose_band", "decompose",
    "wl_band_of_layer", "wl_device_status",
    "wl_last_error", "wl_version", "wl_selftest_wait", "WLStack", "EXPORTED_SYMBOLS", "WL_OK", "WL_ERR_INVALID_ARG",
    "KVCache", "CacheSeqs", "RopeTable", "wl_rope_append", "wl_cache_read", "wl_tree_attention",
    "wl_tree_attention_workspace_bytes", "wl_norm_residual",
    "F8Weight", "PagePool", "wl_quant_f8", "wl_linear_f8", "wl_verify", "wl_page_plan",
    "WL_ERR_UNSUPPORTED", "WL_ERR_CUDA", "WL_ERR_TIMEOUT", "WL_ERR_WORKSPACE", "WL_ERR_INTERNAL", "WL_MAX_RANK",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libwl.so")

WL_OK, WL_ERR_INVALID_ARG, WL_ERR_UNSUPPORTED, WL_ERR_CUDA, WL_ERR_TIMEOUT, WL_ERR_WORKSPACE, WL_ERR_INTERNAL = range(7)
WL_OUT_BF16, WL_OUT_F32 = 0, 1
WL_MAX_RANK = 128
STATUS_NAMES = {0: "WL_OK", 1: "WL_ERR_INVALID_ARG", 2: "WL_ERR_UNSUPPORTED", 3: "WL_ERR_CUDA",
                4: "WL_ERR_TIMEOUT", 5: "WL_ERR_WORKSPACE", 6: "WL_ERR_INTERNAL"}

# Every function include/wl.h declares.
EXPORTED_SYMBOLS = ("wl_linear", "wl_qkv_fused", "wl_linear_f32", "wl_qkv_fused_f32", "wl_decompose_workspace_bytes",
                    "wl_decompose_band", "wl_mlp_workspace_bytes", "wl_mlp_geglu_fused",
                    "wl_mlp_geglu_fused_noalloc", "wl_materialize", "wl_stack_create", "wl_stack_decode",
                    "wl_stack_destroy", "wl_rope_phases", "wl_rope_append", "wl_cache_read",
                    "wl_tree_attention_workspace_bytes", "wl_tree_attention", "wl_norm_residual", "wl_quant_f8", "wl_linear_f8",
                    "wl_verify", "wl_page_plan", "wl_band_of_layer", "wl_device_status", "wl_last_error", "wl_version", "wl_selftest_wait")


class WLError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class _Proj(C.Structure):
    _fields_ = [("W0", C.c_void_p), ("s", C.c_void_p), ("U", C.c_void_p), ("V", C.c_void_p),
                ("out", C.c_int64)]


class _ProjF32(C.Structure):
    _fields_ = [("W0", C.c_void_p), ("s", C.c_void_p), ("U", C.c_void_p), ("V", C.c_void_p),
                ("out", C.c_int64)]


class _Layer(C.Structure):
    _fields_ = [(n, _Proj) for n in ("q", "k", "v", "o", "gate", "up", "down")]


class _LayerOut(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("yq", "yk", "yv", "yo", "ym")]


class _Cache(C.Structure):
    _fields_ = ([(n, C.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, C.c_int64) for n in ("pages", "kv_heads", "page_size", "dim")] + [("format", C.c_int)])


class _Seqs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("pages", "len", "count")] + [(n, C.c_int64) for n in ("batch", "max_pages", "n")]


class _Rope(C.Structure):
    _fields_ = [("phase", C.c_void_p), ("rot", C.c_int64), ("interleaved", C.c_int32), ("amplitude", C.c_float)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libwl.so (built in-tree by build.py); raise if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"libwl.so not found at {_LIB_PATH}; build it with "
                "`python -m rank_weight_reconstruction_wl_gb300.build` (needs nvcc)")
        L = C.CDLL(_LIB_PATH)
        i64, vp, st = C.c_int64, C.c_void_p, C.c_int
        L.wl_linear.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, C.c_int, vp]
        L.wl_linear.restype = st
        L.wl_qkv_fused.argtypes = [vp, _Proj, _Proj, _Proj, vp, vp, vp, i64, i64, i64, C.c_int, vp]
        L.wl_qkv_fused.restype = st
        L.wl_linear_f32.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, C.c_int, vp]
        L.wl_linear_f32.restype = st
        L.wl_qkv_fused_f32.argtypes = [vp, _ProjF32, _ProjF32, _ProjF32, vp, vp, vp, i64, i64, i64, C.c_int, vp]
        L.wl_qkv_fused_f32.restype = st
        L.wl_decompose_workspace_bytes.argtypes = [i64, i64, i64, i64]
        L.wl_decompose_workspace_bytes.restype = C.c_size_t
        L.wl_decompose_band.argtypes = [C.POINTER(C.c_void_p), i64, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp,
                                        C.c_size_t, vp]
        L.wl_decompose_band.restype = st
        L.wl_mlp_workspace_bytes.argtypes = [i64, i64, i64, i64, C.c_int]
        L.wl_mlp_workspace_bytes.restype = C.c_size_t
        L.wl_mlp_geglu_fused.argtypes = [vp, _Proj, _Proj, _Proj, vp, i64, i64, i64, i64, vp,
                                         C.c_size_t, C.c_int, vp]
        L.wl_mlp_geglu_fused.restype = st
        L.wl_mlp_geglu_fused_noalloc.argtypes = [vp, _Proj, _Proj, _Proj, vp, i64, i64, i64, i64,
                                                 C.c_int, vp]
        L.wl_mlp_geglu_fused_noalloc.restype = st
        L.wl_materialize.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, C.c_int, vp]
        L.wl_materialize.restype = st
        L.wl_stack_create.argtypes = [C.POINTER(C.c_void_p), C.POINTER(_Layer), C.POINTER(_LayerOut),
                                      i64, i64, i64, i64]
        L.wl_stack_create.restype = st
        L.wl_stack_decode.argtypes = [vp, vp, vp]
        L.wl_stack_decode.restype = st
        L.wl_stack_destroy.argtypes = [vp]
        L.wl_stack_destroy.restype = None
        f64, f32 = C.c_double, C.c_float
        L.wl_rope_phases.argtypes = [i64, f64, C.c_int, f64, f64, f64, f64, C.POINTER(C.c_uint64), C.POINTER(f32)]
        L.wl_rope_phases.restype = st
        L.wl_rope_append.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, C.c_int, vp, _Rope, _Cache, _Seqs, vp]
        L.wl_rope_append.restype = st
        L.wl_cache_read.argtypes = [_Cache, _Seqs, vp, vp, C.c_int, vp]
        L.wl_cache_read.restype = st
        L.wl_tree_attention_workspace_bytes.argtypes = [i64] * 5
        L.wl_tree_attention_workspace_bytes.restype = C.c_size_t
        L.wl_tree_attention.argtypes = [vp, i64, vp, f32, _Cache, _Seqs, vp, vp, C.c_size_t, vp]
        L.wl_tree_attention.restype = st
        L.wl_norm_residual.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, i64, i64, f32, f32, f32, f32, C.c_int, C.c_int,
                                       C.c_int, vp]
        L.wl_norm_residual.restype = st
        L.wl_quant_f8.argtypes = [vp, i64, C.c_int, i64, i64, i64, vp, vp, vp]
        L.wl_quant_f8.restype = st
        L.wl_linear_f8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, C.c_int, vp]
        L.wl_linear_f8.restype = st
        L.wl_verify.argtypes = [vp, i64, C.c_int, vp, i64, C.c_int, vp, vp, vp, vp, vp, f64, i64, i64, i64, vp, vp, vp, vp]
        L.wl_verify.restype = st
        L.wl_page_plan.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp]
        L.wl_page_plan.restype = st
        L.wl_band_of_layer.argtypes = [i64, i64, i64]
        L.wl_band_of_layer.restype = i64
        L.wl_device_status.argtypes = [vp]
        L.wl_device_status.restype = st
        L.wl_selftest_wait.argtypes = [vp]
        L.wl_selftest_wait.restype = st
        L.wl_last_error.restype = C.c_char_p
        L.wl_version.restype = C.c_char_p
        _lib = L
        return L


# ------------------------------------------------------------ marshalling --
def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _one_device(t, name: str, index):
    """Refuses a tensor of another device than `index` (None: any)."""
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _theta(th):
    if isinstance(th, (tuple, list)):
        return tuple(th)
    return th.W0, th.s, th.U, th.V


def _proj(th, inp: int, r: int, name: str):
    W0, s, U, V = _theta(th)
    out = W0.shape[0]
    _need(W0, f"{name}.W0", torch.bfloat16, (out, inp))
    _need(s, f"{name}.s", torch.float32, (out,))
    if r > 0:
        _need(U, f"{name}.U", torch.bfloat16, (out, r))
        _need(V, f"{name}.V", torch.bfloat16, (inp, r))
    return _Proj(W0.data_ptr(), s.data_ptr(), U.data_ptr() if r > 0 else None,
                 V.data_ptr() if r > 0 else None, out)


def _proj_f32(th, inp: int, r: int, name: str):
    W0, s, U, V = _theta(th)
    out = W0.shape[0]
    _need(W0, f"{name}.W0", torch.float32, (out, inp))
    _need(s, f"{name}.s", torch.float32, (out,))
    if r > 0:
        _need(U, f"{name}.U", torch.float32, (out, r))
        _need(V, f"{name}.V", torch.float32, (inp, r))
    return _ProjF32(W0.data_ptr(), s.data_ptr(), U.data_ptr() if r > 0 else None,
                    V.data_ptr() if r > 0 else None, out)


def _rank(th) -> int:
    U = _theta(th)[2]
    return 0 if U is None else int(U.shape[1])


def _ydt(dtype) -> int:
    if dtype is torch.bfloat16:
        return WL_OUT_BF16
    if dtype is torch.float32:
        return WL_OUT_F32
    if dtype in (torch.bfloat16, "bf16"):
        return WL_OUT_BF16
    if dtype in (torch.float32, "f32", "fp32"):
        return WL_OUT_F32
    raise ValueError(f"output dtype must be bfloat16 or float32, got {dtype}")


def _tdt(ydt: int):
    return torch.float32 if ydt == WL_OUT_F32 else torch.bfloat16


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _stream_object(stream, device):
    """The torch stream of a call (None: the current one, which torch.cuda.stream() leaves as it is)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device)


def _empty(shape, dtype, device, stream):
    """A new tensor of the stream that the call runs on (None: the current one).
    Of another stream's pool it could be a block that queued work of that stream
    still uses, and the allocator would hand it on without waiting for the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(status: int):
    if status != WL_OK:
        raise WLError(status, lib().wl_last_error().decode())


# -------------------------------------------------------------------- API --
def wl_linear(x, W0, s, U, V, y=None, ydt=torch.bfloat16, stream=None):
    """y = s*(x W0^T) + (x V) U^T  (x [T,in] -> y [T,out] bf16/fp32).

    bf16 x and bundle: wl_linear; fp32 x and bundle (the fp32 encoding):
    wl_linear_f32."""
    T, inp = x.shape
    out = W0.shape[0]
    r = 0 if U is None else int(U.shape[1])
    code = _ydt(ydt)
    if x.dtype == torch.float32:
        p = _proj_f32((W0, s, U, V), inp, r, "theta")
        if y is None:
            y = _empty((T, out), _tdt(code), x.device, stream)
        _need(x, "x", torch.float32)
        _need(y, "y", _tdt(code), (T, out))
        with torch.cuda.device(x.device):
            _check(lib().wl_linear_f32(_ptr(x), p.W0, p.s, p.U, p.V, _ptr(y), T, inp, out, r, code,
                                       _stream(stream, x.device)))
        return y
    _need(x, "x", torch.bfloat16)
    p = _proj((W0, s, U, V), inp, r, "theta")
    if y is None:
        y = _empty((T, out), _tdt(code), x.device, stream)
    _need(y, "y", _tdt(code), (T, out))
    with torch.cuda.device(x.device):
        _check(lib().wl_linear(_ptr(x), p.W0, p.s, p.U, p.V, _ptr(y), T, inp, out, r, code,
                               _stream(stream, x.device)))
    return y


def wl_qkv_fused(x, q, k, v, outs=None, ydt=torch.bfloat16, stream=None):
    """Q/K/V projections of one x in one launch; returns (yq, yk, yv)."""
    T, inp = x.shape
    r = _rank(q)
    code = _ydt(ydt)
    if x.dtype == torch.float32:
        _need(x, "x", torch.float32)
        ps = [_proj_f32(th, inp, r, n) for th, n in ((q, "q"), (k, "k"), (v, "v"))]
        if outs is None:
            outs = tuple(_empty((T, p.out), _tdt(code), x.device, stream) for p in ps)
        for o, p, n in zip(outs, ps, ("yq", "yk", "yv")):
            _need(o, n, _tdt(code), (T, p.out))
        with torch.cuda.device(x.device):
            _check(lib().wl_qkv_fused_f32(_ptr(x), ps[0], ps[1], ps[2], _ptr(outs[0]), _ptr(outs[1]),
                                          _ptr(outs[2]), T, inp, r, code, _stream(stream, x.device)))
        return tuple(outs)
    _need(x, "x", torch.bfloat16)
    ps = [_proj(th, inp, r, n) for th, n in ((q, "q"), (k, "k"), (v, "v"))]
    if outs is None:
        outs = tuple(_empty((T, p.out), _tdt(code), x.device, stream) for p in ps)
    for o, p, n in zip(outs, ps, ("yq", "yk", "yv")):
        _need(o, n, _tdt(code), (T, p.out))
    with torch.cuda.device(x.device):
        _check(lib().wl_qkv_fused(_ptr(x), ps[0], ps[1], ps[2], _ptr(outs[0]), _ptr(outs[1]),
                                  _ptr(outs[2]), T, inp, r, code, _stream(stream, x.device)))
    return tuple(outs)


def wl_mlp_workspace_bytes(T, hidden, inter, r, ydt=torch.bfloat16) -> int:
    return int(lib().wl_mlp_workspace_bytes(T, hidden, inter, r, _ydt(ydt)))


_ws_cache: dict = {}


def mlp_workspace(T, hidden, inter, r, ydt=torch.bfloat16, device=None) -> torch.Tensor:
    """A zeroed workspace of the right size (cached per device and size)."""
    n = wl_mlp_workspace_bytes(T, hidden, inter, r, ydt)
    if n == 0:
        raise ValueError("invalid MLP sizes")
    dev = torch.device(device if device is not None else "cuda")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    key = (dev.index, n)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.zeros(n + 256, dtype=torch.uint8, device=dev)
        off = (-ws.data_ptr()) % 256
        ws = ws[off:off + n]
        _ws_cache[key] = ws
    return ws


def wl_mlp_geglu_fused(x, gate, up, down, y=None, workspace=None, ydt=torch.bfloat16,
                       stream=None):
    """y = (gelu_tanh(x Wg^T) * (x Wu^T)) Wd^T with every W a weightless projection."""
    T, hidden = x.shape
    r = _rank(gate)
    inter = _theta(gate)[0].shape[0]
    code = _ydt(ydt)
    _need(x, "x", torch.bfloat16)
    pg = _proj(gate, hidden, r, "gate")
    pu = _proj(up, hidden, r, "up")
    pd = _proj(down, inter, r, "down")
    if y is None:
        y = _empty((T, hidden), _tdt(code), x.device, stream)
    _need(y, "y", _tdt(code), (T, hidden))
    if workspace is None:
        workspace = mlp_workspace(T, hidden, inter, r, ydt, x.device)
    with torch.cuda.device(x.device):
        _check(lib().wl_mlp_geglu_fused(_ptr(x), pg, pu, pd, _ptr(y), T, hidden, inter, r,
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        code, _stream(stream, x.device)))
    return y


def wl_mlp_geglu_fused_noalloc(x, gate, up, down, y, ydt=torch.bfloat16, stream=None):
    """Same MLP without a caller workspace (library's built-in 4 MiB scratch),
    for callers that cannot allocate device memory.  `y` must be given."""
    T, hidden = x.shape
    r = _rank(gate)
    inter = _theta(gate)[0].shape[0]
    code = _ydt(ydt)
    _need(x, "x", torch.bfloat16)
    pg = _proj(gate, hidden, r, "gate")
    pu = _proj(up, hidden, r, "up")
    pd = _proj(down, inter, r, "down")
    _need(y, "y", _tdt(code), (T, hidden))
    with torch.cuda.device(x.device):
        _check(lib().wl_mlp_geglu_fused_noalloc(_ptr(x), pg, pu, pd, _ptr(y), T, hidden, inter, r,
                                                code, _stream(stream, x.device)))
    return y


def wl_materialize(W0, s, U, V, dt=torch.bfloat16, out=None, stream=None):
    """W_eff = s*W0 + U V^T, bit-exact fixed fp32 order, as bf16 or fp32."""
    o, inp = W0.shape
    r = 0 if U is None else int(U.shape[1])
    code = _ydt(dt)
    p = _proj((W0, s, U, V), inp, r, "theta")
    if out is None:
        out = _empty((o, inp), _tdt(code), W0.device, stream)
    _need(out, "W_eff", _tdt(code), (o, inp))
    with torch.cuda.device(W0.device):
        _check(lib().wl_materialize(p.W0, p.s, p.U, p.V, _ptr(out), o, inp, r, code,
                                    _stream(stream, W0.device)))
    return out


def wl_decompose_band(Ws, r, p=8, iters=4, omega=None, seed=0, stream=None):
    """The theta bundle of one band: Ws (list of n bf16 [out, in] weights of
    one projection family, sharing one W0) -> (W0 [out, in] bf16, s [n, out]
    fp32, U [n, out, r] bf16, V [n, in, r] bf16).  omega [in, r + p] fp32 is
    the Gaussian start of the subspace iteration (drawn from `seed` when not
    given).  The binding allocates the outputs and the workspace; the library
    call allocates nothing."""
    n = len(Ws)
    out, inp = Ws[0].shape
    dev = Ws[0].device
    for i, W in enumerate(Ws):
        _need(W, f"Ws[{i}]", torch.bfloat16, (out, inp))
    k = r + p
    if omega is None:
        g = torch.Generator(device=dev)
        g.manual_seed(int(seed))
        with torch.cuda.stream(_stream_object(stream, dev)):
            omega = torch.randn(inp, k, generator=g, device=dev, dtype=torch.float32)
    if r > 0:
        _need(omega, "omega", torch.float32, (inp, k))
    W0 = _empty((out, inp), torch.bfloat16, dev, stream)
    s = _empty((n, out), torch.float32, dev, stream)
    U = _empty((n, out, r), torch.bfloat16, dev, stream)
    V = _empty((n, inp, r), torch.bfloat16, dev, stream)
    # 0 for sizes the library rejects: the call below then reports why
    nb = int(lib().wl_decompose_workspace_bytes(out, inp, r, p))
    ws = _empty(nb + 256, torch.uint8, dev, stream)
    off = (-ws.data_ptr()) % 256
    ptrs = (C.c_void_p * n)(*[W.data_ptr() for W in Ws])
    with torch.cuda.device(dev):
        _check(lib().wl_decompose_band(ptrs, n, out, inp, r, p, iters, _ptr(omega) if r > 0 else None, _ptr(W0),
                                       _ptr(s), _ptr(U) if r > 0 else None, _ptr(V) if r > 0 else None,
                                       C.c_void_p(ws.data_ptr() + off), nb, _stream(stream, dev)))
    return W0, s, U, V


def decompose(Ws, G, r, p=8, iters=4, seed=0, stream=None):
    """Theta bundles of a family's L dense weights with G shared W0 blocks:
    layer l uses block wl_band_of_layer(l, L, G).  Returns a list of L
    (W0, s, U, V) tuples; layers of a band share their W0 tensor."""
    L = len(Ws)
    bands = [[] for _ in range(G)]
    for l in range(L):
        bands[wl_band_of_layer(l, L, G)].append(l)
    res = [None] * L
    for b, members in enumerate(bands):
        W0, s, U, V = wl_decompose_band([Ws[l] for l in members], r, p, iters, seed=seed + b, stream=stream)
        for j, l in enumerate(members):
            res[l] = (W0, s[j], U[j], V[j])
    return res


class WLStack:
    """A stack of weightless decoder layers run by one launch per step
    (wl_stack_create / wl_stack_decode).

    layers: objects with q, k, v, o, gate, up, down theta bundles (all bf16
    W0, U, V and fp32 s on one device).  The stack owns one set of bf16 output
    buffers per layer, ``outs[l] = {"yq", "yk", "yv", "yo", "ym"}``;
    ``decode(x)`` writes all of them and returns ``outs[-1]["ym"]``.
    Raises WLError (WL_ERR_UNSUPPORTED) for sizes the stack kernels do not
    take (T > 32, r > 32, hidden / q.out / gate.out not multiples of 64).
    """

    def __init__(self, layers, T: int, device=None):
        self.dev = torch.device(device) if device is not None else layers[0].q.W0.device
        self.T = int(T)
        th0 = layers[0]
        self.hidden = int(th0.q.W0.shape[1])
        self.r = _rank(th0.q)
        qd, kd, vd = th0.q.W0.shape[0], th0.k.W0.shape[0], th0.v.W0.shape[0]
        inter = th0.gate.W0.shape[0]
        h, r = self.hidden, self.r
        L = len(layers)
        z = dict(dtype=torch.bfloat16, device=self.dev)
        self.outs = [{"yq": torch.empty(T, qd, **z), "yk": torch.empty(T, kd, **z),
                      "yv": torch.empty(T, vd, **z), "yo": torch.empty(T, h, **z),
                      "ym": torch.empty(T, h, **z)} for _ in range(L)]
        self._layers = (_Layer * L)()
        self._louts = (_LayerOut * L)()
        self._keep = layers  # the stack refers to the layers' device memory
        for l, th in enumerate(layers):
            ly = self._layers[l]
            ly.q = _proj(th.q, h, r, f"layer {l} q")
            ly.k = _proj(th.k, h, r, f"layer {l} k")
            ly.v = _proj(th.v, h, r, f"layer {l} v")
            ly.o = _proj(th.o, qd, r, f"layer {l} o")
            ly.gate = _proj(th.gate, h, r, f"layer {l} gate")
            ly.up = _proj(th.up, h, r, f"layer {l} up")
            ly.down = _proj(th.down, inter, r, f"layer {l} down")
            o = self.outs[l]
            self._louts[l] = _LayerOut(o["yq"].data_ptr(), o["yk"].data_ptr(), o["yv"].data_ptr(),
                                       o["yo"].data_ptr(), o["ym"].data_ptr())
        self._h = C.c_void_p()
        with torch.cuda.device(self.dev):
            _check(lib().wl_stack_create(C.byref(self._h), self._layers, self._louts, L, self.T, h, r))

    @property
    def out(self) -> torch.Tensor:
        return self.outs[-1]["ym"]

    def decode(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        _need(x, "x", torch.bfloat16, (self.T, self.hidden))
        with torch.cuda.device(self.dev):
            _check(lib().wl_stack_decode(self._h, _ptr(x), _stream(stream, self.dev)))
        return self.out

    def close(self):
        if self._h:
            lib().wl_stack_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------- decoder-layer operators --
class RopeTable:
    """Rotary table: ``phases`` [rot/2] int64 on the GPU (turns per position in
    units of 2^-64 turn), the pair layout and the amplitude of cos and sin."""

    SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}

    def __init__(self, phases: torch.Tensor, interleaved: bool = False, amplitude: float = 1.0):
        _need(phases, "phases", torch.int64)
        self.phases, self.interleaved, self.amplitude = phases, bool(interleaved), float(amplitude)
        self.rot = 2 * phases.numel()
        self.index = phases.get_device()
        self._c = _Rope(phases.data_ptr(), self.rot, int(self.interleaved), self.amplitude)

    @classmethod
    def make(cls, rot: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
             orig_len: float = 0.0, fast: float = 32.0, slow: float = 1.0, device="cuda") -> "RopeTable":
        """The table of wl_rope_phases, copied to the device.  scaling: "none",
        "linear" (f/factor), "base" (a larger base) or "ramp" (both, by how
        often a pair turns in orig_len positions)."""
        phases, amplitude = rope_phases(rot, base, scaling, factor, orig_len, fast, slow)
        return cls(phases.to(device), interleaved, amplitude)


def rope_phases(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, orig_len: float = 0.0,
                fast: float = 32.0, slow: float = 1.0):
    """(phases [rot/2] int64 on the host, amplitude) of wl_rope_phases."""
    if scaling not in RopeTable.SCALINGS:
        raise ValueError(f"unknown rotary scaling {scaling!r}")
    ph = (C.c_uint64 * max(1, int(rot) // 2))()
    amp = C.c_float()
    _check(lib().wl_rope_phases(int(rot), base, RopeTable.SCALINGS[scaling], factor, orig_len, fast, slow, ph, C.byref(amp)))
    return torch.tensor([C.c_int64(v).value for v in ph[:int(rot) // 2]], dtype=torch.int64), amp.value


class KVCache:
    """A paged key/value cache: k, v [pages, kv_heads, page_size, dim]
    (float8_e4m3fn or bfloat16 codes) and fp32 row scales k_scale, v_scale
    [pages, kv_heads, page_size]; a value is code * scale."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a tensor [pages, kv_heads, page_size, dim]")
        if k.dtype not in (torch.float8_e4m3fn, torch.bfloat16):
            raise TypeError(f"a cache holds float8_e4m3fn or bfloat16, got {k.dtype}")
        _need(k, "k", k.dtype)
        _need(v, "v", k.dtype, k.shape)
        _need(k_scale, "k_scale", torch.float32, k.shape[:3])
        _need(v_scale, "v_scale", torch.float32, k.shape[:3])
        if not (k.device == v.device == k_scale.device == v_scale.device):
            raise ValueError("the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.index = k.device, k.get_device()
        self.pages, self.kv_heads, self.page_size, self.dim = (int(n) for n in k.shape)
        self._c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.pages, self.kv_heads,
                         self.page_size, self.dim, 0 if k.dtype == torch.float8_e4m3fn else 1)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int, dim: int, dtype=torch.float8_e4m3fn, device="cuda") -> "KVCache":
        """A cache of unwritten pages."""
        shape = (pages, kv_heads, page_size, dim)
        if dtype not in (torch.float8_e4m3fn, torch.bfloat16):
            raise TypeError(f"a cache holds float8_e4m3fn or bfloat16, got {dtype}")
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        ks, vs = (torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


class CacheSeqs:
    """The sequences of a call: pages [batch, max_pages] int32 (page of each run
    of page_size positions), len [batch] int32 (positions already in the
    cache), n new positions each, or count[b] <= n of them (int32).  All on the
    GPU and read when the kernels run, so they may change between calls."""

    def __init__(self, pages: torch.Tensor, len: torch.Tensor, n: int, count: torch.Tensor | None = None):
        _need(pages, "pages", torch.int32)
        if pages.dim() != 2:
            raise ValueError("pages must be [batch, max_pages]")
        B = int(pages.shape[0])
        _need(len, "len", torch.int32, (B,))
        if count is not None:
            _need(count, "count", torch.int32, (B,))
        if pages.device != len.device or (count is not None and pages.device != count.device):
            raise ValueError("pages, len and count must be on one device")
        self.index = pages.get_device()
        self.pages, self.len, self.n, self.count, self.batch = pages, len, int(n), count, B
        self.tokens = B * self.n
        self._c = _Seqs(pages.data_ptr(), len.data_ptr(), None if count is None else count.data_ptr(), B,
                        int(pages.shape[1]), self.n)


def _token_rows(t, name: str, dtype, tokens: int, width: int, index=None) -> int:
    """Row stride in elements of a tensor of `tokens` rows of `width` elements:
    [tokens, width], [tokens, heads, dim] or [batch, n, heads, dim], rows any
    one distance apart; on device `index` (None: any CUDA device)."""
    if t.__class__ is torch.Tensor and t.dtype is dtype and t.get_device() == index and t.is_contiguous() and t.numel() == tokens * width:
        return width
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _one_device(t, name, index)
    if t.numel() != tokens * width:
        raise ValueError(f"{name} must hold {tokens} rows of {width} elements, got {tuple(t.shape)}")
    if t.is_contiguous():
        return width
    sh, sd = t.shape, t.stride()
    lead = 2 if t.dim() == 4 else 1
    run = 1  # the trailing dimensions are one run of `width` elements
    for n, st in zip(reversed(sh[lead:]), reversed(sd[lead:])):
        if n > 1 and st != run:
            raise ValueError(f"{name}: each token's row must be contiguous")
        run *= n
    if run != width or t.dim() not in (2, 3, 4):
        raise ValueError(f"{name} must be [tokens, heads*dim], [tokens, heads, dim] or [batch, n, heads, dim]")
    if lead == 2 and sh[0] > 1 and sh[1] > 1 and sd[0] != sh[1] * sd[1]:
        raise ValueError(f"{name}: all token rows must be the same distance apart")
    return int(sd[lead - 1]) if sh[lead - 1] > 1 else int(sd[0]) if lead == 2 and sh[0] > 1 else width


# The calls below are as short as their launches (a few microseconds), so the
# binding keeps its own share small: one pass over the arguments, and the
# current device and stream by torch's cheapest queries.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _checked(t, name: str, dtype, shape, index) -> int:
    """The address of a contiguous tensor of this type and shape (None: any) on device `index`."""
    if t.__class__ is torch.Tensor and t.dtype is dtype and t.get_device() == index and (shape is None or t.shape == shape) and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype, shape)
    _one_device(t, name, index)
    return t.data_ptr()


def _on_device(fn, device, args):
    """fn(*args) where another device than `device` is the current one."""
    with torch.cuda.device(device):
        return fn(*args)


def _stream_of(index: int, stream) -> int:
    if stream is None:
        return _current_stream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _run(fn, device, stream, *args):
    """fn(*args, stream) on `device`; raises what it reports."""
    index = device.index
    st = _current_stream(index) if stream is None else _stream_of(index, stream)
    status = fn(*args, st) if _current_device() == index else _on_device(fn, device, (*args, st))
    if status:
        _check(status)


_NO_ROPE = _Rope(None, 0, 0, 1.0)
_OTHER_SEQS = "the sequences must be on the cache's device"


def wl_rope_append(q, k, v, positions, rope: RopeTable | None, cache: KVCache, seqs: CacheSeqs, q_out=None, stream=None):
    """Rotates q and k and writes k and v to the cache, quantised, at positions
    len[b] .. len[b] + count[b] - 1; returns q_out, the rotated q as bf16 (None
    where q is None).  q, k, v: the outputs of wl_qkv_fused, or any bf16 or
    fp32 tensors of batch * n token rows (_token_rows).  positions: int32
    [batch, n], or None for len[b] + i.  rope None: no rotation."""
    dt = k.dtype
    code = _ydt(dt)
    tokens, dim, index = seqs.tokens, cache.dim, cache.index
    if seqs.index != index:
        raise ValueError(_OTHER_SEQS)
    kvw = cache.kv_heads * dim
    ks, vs = _token_rows(k, "k", dt, tokens, kvw, index), _token_rows(v, "v", dt, tokens, kvw, index)
    heads, qs, qp, op = 0, 0, None, None
    if q is not None:
        heads = q.numel() // max(1, tokens * dim)
        qs = _token_rows(q, "q", dt, tokens, heads * dim, index)
        qp = q.data_ptr()
        if q_out is None:
            q_out = _empty(q.shape, torch.bfloat16, q.device, stream)
            op = q_out.data_ptr()
        else:
            op = _checked(q_out, "q_out", torch.bfloat16, q.shape, index)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    pp = None
    if positions is not None:
        pp = _checked(positions, "positions", torch.int32, None, index)
        if positions.numel() != tokens:
            raise ValueError(f"positions must hold batch * n = {tokens} numbers, got {tuple(positions.shape)}")
    if rope is not None and rope.index != index:
        raise ValueError(f"the rotary table must be on the cache's device, cuda:{index}")
    _run((_lib or lib()).wl_rope_append, cache.device, stream, qp, k.data_ptr(), v.data_ptr(), op, heads, qs, ks, vs, code, pp,
         _NO_ROPE if rope is None else rope._c, cache._c, seqs._c)
    return q_out


def wl_cache_read(cache: KVCache, seqs: CacheSeqs, dt=torch.bfloat16, outs=None, stream=None):
    """The cache's values at positions len[b] + i, i < count[b] (zeros beyond):
    (k, v) [batch, n, kv_heads, dim] as bf16 or fp32."""
    code = _ydt(dt)
    td, index = _tdt(code), cache.index
    if seqs.index != index:
        raise ValueError(_OTHER_SEQS)
    shape = (seqs.batch, seqs.n, cache.kv_heads, cache.dim)
    if outs is None:
        outs = (_empty(shape, td, cache.device, stream), _empty(shape, td, cache.device, stream))
        kp, vp = outs[0].data_ptr(), outs[1].data_ptr()
    else:
        kp, vp = _checked(outs[0], "k_out", td, shape, index), _checked(outs[1], "v_out", td, shape, index)
    _run((_lib or lib()).wl_cache_read, cache.device, stream, cache._c, seqs._c, kp, vp, code)
    return tuple(outs)


def wl_tree_attention_workspace_bytes(batch, n, q_heads, kv_heads, dim) -> int:
    return int(lib().wl_tree_attention_workspace_bytes(batch, n, q_heads, kv_heads, dim))


def wl_tree_attention(q, cache: KVCache, seqs: CacheSeqs, mask=None, scale: float | None = None, out=None, workspace=None,
                      stream=None):
    """Attention of the n newest tokens of each sequence over its cache; token i
    sees the len[b] positions before them and the new tokens j with bit j of
    mask[b, i] (int64; None: 0..i).  q bf16 [batch, n, q_heads, dim] (or
    [batch * n, q_heads * dim]) -> out of the same shape.  scale defaults to
    dim ** -0.5.  workspace: at least wl_tree_attention_workspace_bytes() bytes,
    256-byte aligned; by default allocated for the call."""
    tokens, dim, index = seqs.tokens, cache.dim, cache.index
    if seqs.index != index:
        raise ValueError(_OTHER_SEQS)
    qp = _checked(q, "q", torch.bfloat16, None, index)
    heads = q.numel() // max(1, tokens * dim)
    if heads * tokens * dim != q.numel():
        raise ValueError(f"q must hold batch * n = {tokens} rows of heads * {dim} elements, got {tuple(q.shape)}")
    mp = None
    if mask is not None:
        mp = _checked(mask, "mask", torch.int64, None, index)
        if mask.numel() != tokens:
            raise ValueError(f"mask must hold batch * n = {tokens} words, got {tuple(mask.shape)}")
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty(q.shape, torch.bfloat16, q.device, stream)
        op = out.data_ptr()
    else:
        op = _checked(out, "out", torch.bfloat16, q.shape, index)
    L = _lib or lib()
    if workspace is None:
        nb = max(256, L.wl_tree_attention_workspace_bytes(seqs.batch, seqs.n, heads, cache.kv_heads, dim))
        workspace = _empty(nb, torch.uint8, cache.device, stream)
        ws = workspace.data_ptr()
    else:
        ws = _checked(workspace, "workspace", getattr(workspace, "dtype", None), None, index)
    _run(L.wl_tree_attention, cache.device, stream, qp, heads, mp, dim ** -0.5 if scale is None else scale, cache._c, seqs._c, op,
         ws, workspace.numel() * workspace.element_size())
    return out


def wl_norm_residual(y, x, w_post=None, w_pre=None, gate=None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                     w_offset: float = 0.0, x_out=None, h_dt=torch.bfloat16, h=None, stream=None):
    """x' = alpha x + beta gate (rms(y) (w_offset + w_post)) and h = rms(x')
    (w_offset + w_pre): the norm after one block, its gate, the residual and the
    norm before the next, in one launch.  y [T, H] or None; gate [T, H], or [H]
    or [1, H] for all tokens, of y's type; w_post, w_pre fp32 [H] or None (no
    norm after the block; no h).  Returns (x', h); x_out may be x (in place)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [T, H]")
    shape = x.shape
    T, H = shape
    dt = x.dtype
    xc = yc = _ydt(dt)
    index = x.get_device() if x.is_cuda else None
    xp = _checked(x, "x", dt, shape, index)
    yp = gp = wp = wq = xo = hp = None
    gs = 0
    if y is not None:
        yc = _ydt(y.dtype)
        yp = _checked(y, "y", y.dtype, shape, index)
    if gate is not None:
        if y is None:
            raise ValueError("gate needs y")
        gp = _checked(gate, "gate", y.dtype, None, index)
        if gate.numel() != H:
            if gate.shape != shape:
                raise ValueError(f"gate must be [{T}, {H}], [1, {H}] or [{H}], got {tuple(gate.shape)}")
            gs = H
    if w_post is not None:
        wp = _checked(w_post, "w_post", torch.float32, (H,), index)
    if w_pre is not None:
        wq = _checked(w_pre, "w_pre", torch.float32, (H,), index)
    if x_out is not None:
        xo = _checked(x_out, "x_out", dt, shape, index)
    elif y is not None or alpha != 1.0:
        x_out = torch.empty_like(x) if stream is None else _empty(shape, dt, x.device, stream)
        xo = x_out.data_ptr()
    hc = _ydt(h_dt)
    td = _tdt(hc)
    if h is not None:
        hp = _checked(h, "h", td, shape, index)
    elif w_pre is not None:
        if stream is not None:
            h = _empty(shape, td, x.device, stream)
        else:
            h = torch.empty_like(x) if td is dt else torch.empty_like(x, dtype=td)
        hp = h.data_ptr()
    _run((_lib or lib()).wl_norm_residual, x.device, stream, yp, gp, gs, xp, wp, wq, xo, hp, T, H, alpha, beta, eps, w_offset, yc,
         xc, hc)
    return (x if x_out is None else x_out), h


# ------------------------- operators between a step's last states and the next --
_F8 = torch.float8_e4m3fn


def _rows_of(t, name: str, dtype, rows: int, width: int, index) -> int:
    """Row stride in elements of a matrix [rows, width] on device `index` whose rows are contiguous."""
    if t.__class__ is torch.Tensor and t.dtype is dtype and t.get_device() == index and t.shape == (rows, width) and t.is_contiguous():
        return width
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _one_device(t, name, index)
    if t.dim() != 2 or tuple(t.shape) != (rows, width):
        raise ValueError(f"{name} must have shape {(rows, width)}, got {tuple(t.shape)}")
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: each row must be contiguous")
    return int(t.stride(0)) if rows > 1 else width


def wl_quant_f8(x, group: int = 1, outs=None, stream=None):
    """e4m3 codes [rows, in] and fp32 scales [ceil(in/128), ceil(rows/group)] of
    x [rows, in] (bf16 or fp32, rows any multiple of 8 elements apart): a
    power-of-two scale for each 128 elements of a row (group 1: activations) or
    each 128 x 128 block (group 128: weights)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [rows, in]")
    rows, inp = x.shape
    code = _ydt(x.dtype)
    index = x.get_device() if x.is_cuda else None
    if index is not None and x.is_contiguous():
        xs = inp
    else:
        xs = _rows_of(x, "x", x.dtype, rows, inp, index)
    shape = (-(-inp // 128), -(-rows // max(1, group)))
    if outs is None:
        codes, scales = _empty((rows, inp), _F8, x.device, stream), _empty(shape, torch.float32, x.device, stream)
        cp, sp = codes.data_ptr(), scales.data_ptr()
    else:
        codes, scales = outs
        cp, sp = _checked(codes, "codes", _F8, (rows, inp), index), _checked(scales, "scales", torch.float32, shape, index)
    _run((_lib or lib()).wl_quant_f8, x.device, stream, x.data_ptr(), xs, code, rows, inp, group, cp, sp)
    return codes, scales


class F8Weight:
    """A dense weight of 8 bits: codes [out, in] float8_e4m3fn and fp32 scales
    [ceil(in/128), ceil(out/128)]; a value is code * scale of its 128 x 128
    block (checkpoints hold the scales transposed)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise ValueError("codes must be a tensor [out, in]")
        _need(codes, "codes", _F8)
        self.out, self.inp = (int(n) for n in codes.shape)
        _need(scales, "scales", torch.float32, (-(-self.inp // 128), -(-self.out // 128)))
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self.codes, self.scales = codes, scales
        self.device, self.index = codes.device, codes.get_device()
        self._cp, self._sp = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def quantise(cls, W: torch.Tensor, stream=None) -> "F8Weight":
        """The nearest such weight to W [out, in] (bf16 or fp32), scales powers of two."""
        return cls(*wl_quant_f8(W, group=128, stream=stream))


def wl_linear_f8(codes, scales, weight: F8Weight, y=None, ydt=torch.bfloat16, stream=None):
    """y = x W^T for x = (codes, scales) of wl_quant_f8 (any fp32 scales
    [ceil(in/128), T]) and an F8Weight; y [T, out] bf16 or fp32."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be a tensor [T, in]")
    index, inp = weight.index, weight.inp
    T = codes.shape[0]
    cp = _checked(codes, "codes", _F8, (T, inp), index)
    sp = _checked(scales, "scales", torch.float32, (-(-inp // 128), T), index)
    code = _ydt(ydt)
    if y is None:
        y = _empty((T, weight.out), _tdt(code), weight.device, stream)
        yp = y.data_ptr()
    else:
        yp = _checked(y, "y", _tdt(code), (T, weight.out), index)
    _run((_lib or lib()).wl_linear_f8, weight.device, stream, cp, sp, weight._cp, weight._sp, yp, T, inp, weight.out, code)
    return y


def wl_verify(logits, tokens, uniforms, mask=None, count=None, draft=None, temperature=1.0, outs=None, stream=None):
    """Which drafted tokens hold, and the token after them: (path [batch, n],
    accepted [batch], next [batch]), int32, as Decoder.accept() takes them.

    logits [batch * n, vocab] bf16 or fp32: row b * n + i is the model's for the
    token after node i of sequence b; tokens int32 [batch, n] (node 0 is known,
    the others are drafted), mask int64 [batch, n] as for wl_tree_attention
    (None: a chain), count int32 [batch] nodes (None: n).  uniforms fp32
    [batch, n] in [0, 1): entry i decides about node i, entry 0 draws the next
    token.  draft [batch * n, vocab] bf16 or fp32: row b * n + u is the
    distribution that node u's children were drawn from; None: they are certain
    (a drafter's best tokens).  temperature: a number or fp32 [batch]; below 1e-6
    the most likely token is taken.  n = 1 is plain sampling.  next is -1, no
    token, where count is 0 (node 0 then still waits, accepted is 0) and where the
    last accepted node's row has no distribution (a NaN, +infinity, all masked)."""
    if not isinstance(tokens, torch.Tensor) or tokens.dim() != 2:
        raise ValueError("tokens must be a tensor [batch, n]")
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a tensor [batch * n, vocab]")
    B, n = tokens.shape
    V = logits.shape[1]
    index = tokens.get_device() if tokens.is_cuda else None
    tp = _checked(tokens, "tokens", torch.int32, None, index)
    ldt = _ydt(logits.dtype)
    ls = _rows_of(logits, "logits", logits.dtype, B * n, V, index)
    up = _checked(uniforms, "uniforms", torch.float32, (B, n), index)
    mp = cp = dp = tt = None
    ddt, ds, temp = WL_OUT_F32, 0, 0.0
    if mask is not None:
        mp = _checked(mask, "mask", torch.int64, (B, n), index)
    if count is not None:
        cp = _checked(count, "count", torch.int32, (B,), index)
    if draft is not None:
        if not isinstance(draft, torch.Tensor):
            raise TypeError("draft must be a torch.Tensor")
        ddt = _ydt(draft.dtype)
        ds = _rows_of(draft, "draft", draft.dtype, B * n, V, index)
        dp = draft.data_ptr()
    if isinstance(temperature, torch.Tensor):
        tt = _checked(temperature, "temperature", torch.float32, (B,), index)
    else:
        temp = float(temperature)
    if outs is None:
        dev = tokens.device
        path, accepted, nxt = (_empty((B, n), torch.int32, dev, stream), _empty((B,), torch.int32, dev, stream),
                               _empty((B,), torch.int32, dev, stream))
        pp, ap, np_ = path.data_ptr(), accepted.data_ptr(), nxt.data_ptr()
    else:
        path, accepted, nxt = outs
        pp = _checked(path, "path", torch.int32, (B, n), index)
        ap, np_ = _checked(accepted, "accepted", torch.int32, (B,), index), _checked(nxt, "next", torch.int32, (B,), index)
    _run((_lib or lib()).wl_verify, tokens.device, stream, logits.data_ptr(), ls, ldt, dp, ds, ddt, tp, up, mp, cp, tt, temp, B, n, V,
         pp, ap, np_)
    return path, accepted, nxt


class PagePool:
    """The free pages of a cache: a stack free[0 .. top - 1] (int32, on the GPU;
    top int32 [1]) of page numbers, pages of page_size positions."""

    def __init__(self, free: torch.Tensor, top: torch.Tensor, page_size: int):
        _need(free, "free", torch.int32)
        if free.dim() != 1:
            raise ValueError("free must be [pages]")
        _need(top, "top", torch.int32, (1,))
        if free.device != top.device:
            raise ValueError("free and top must be on one device")
        self.free, self.top, self.page_size = free, top, int(page_size)
        self.pages = int(free.shape[0])
        self.device, self.index = free.device, free.get_device()

    @classmethod
    def full(cls, pages: int, page_size: int, device="cuda") -> "PagePool":
        """All of `pages` pages free; page 0 is taken first."""
        return cls(torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.full((1,), pages, dtype=torch.int32, device=device), page_size)


def wl_page_plan(pool: PagePool, pages, held, len, n: int = 0, count=None, slots=False, room=None, stream=None):
    """Makes the page table pages [batch, max_pages] (int32) fit len[b] +
    count[b] positions (n new ones each, or count[b] <= n of them): pages past
    them go back to the pool, missing ones are taken, sequences in order, all
    that a sequence misses or none.  held int32 [batch]: how many entries of
    a row are in use.  pages, held and the pool are changed in place.  Returns
    (room, slots): room int32 [batch], how many of the new positions have pages
    (the count of CacheSeqs); slots (True, or an int64 tensor [batch, n]): cache
    row page * page_size + offset of each new position, -1 beyond room."""
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2:
        raise ValueError("pages must be a tensor [batch, max_pages]")
    index, dev = pool.index, pool.device
    B, P = pages.shape
    n = int(n)
    pp = _checked(pages, "pages", torch.int32, None, index)
    hp = _checked(held, "held", torch.int32, (B,), index)
    lp = _checked(len, "len", torch.int32, (B,), index)
    cp = None if count is None else _checked(count, "count", torch.int32, (B,), index)
    if room is None:
        room = _empty((B,), torch.int32, dev, stream)
        rp = room.data_ptr()
    else:
        rp = _checked(room, "room", torch.int32, (B,), index)
    sp = None
    if slots is True:
        slots = _empty((B, n), torch.int64, dev, stream)
        sp = slots.data_ptr()
    elif slots is None or slots is False:
        slots = None
    else:
        sp = _checked(slots, "slots", torch.int64, (B, n), index)
    _run((_lib or lib()).wl_page_plan, dev, stream, pool.free.data_ptr(), pool.top.data_ptr(), pool.pages, pool.page_size, pp, hp, lp, cp,
         B, P, n, rp, sp)
    return room, slots


def wl_band_of_layer(layer: int, L: int, G: int) -> int:
    return int(lib().wl_band_of_layer(layer, L, G))


def wl_device_status(stream=None, device=None) -> int:
    """Synchronise and return (and clear) the device status code."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        return int(lib().wl_device_status(_stream(stream, dev)))


def wl_selftest_wait(stream=None, device=None):
    """Launch the diagnostic kernel whose bounded wait gives up (about 2 s);
    the next wl_device_status() reports WL_ERR_TIMEOUT."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(lib().wl_selftest_wait(_stream(stream, dev)))


def wl_last_error() -> str:
    return lib().wl_last_error().decode()


def wl_version() -> str:
    return lib().wl_version().decode()
