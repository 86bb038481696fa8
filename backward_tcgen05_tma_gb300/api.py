"""Thin Python binding of libswiglu_mlp.so (include/swiglu_mlp.h).

Argument marshalling only: torch supplies device memory (``data_ptr()``) and
the current CUDA stream; every step of the MLP runs in the library's CUDA
kernels.  If the library is missing this module raises -- there is no
fallback path.

The three calls keep the C ABI's names:

* ``swiglu_mlp_fwd(X, Wgu, Wd)``        -> (Y, saved)      saved = [G | U | A]
* ``swiglu_mlp_fwd_nograd(X, Wgu, Wd)`` -> (Y, A)
* ``swiglu_mlp_bwd(dY, X, Wgu, Wd, saved)`` -> (dX, dWgu, dWd); consumes saved

Outputs may be passed in (``out=`` dicts) to avoid allocation.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libswiglu_mlp.so")
# the same library compiled with -DSWIGLU_DEBUG (device index checks)
DEBUG_LIB_PATH = os.path.join(_HERE, "libswiglu_mlp_debug.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "swiglu_mlp.h")

SWIGLU_BF16, SWIGLU_F16, SWIGLU_F32_IEEE = 0, 1, 2
SWIGLU_OP_FWD, SWIGLU_OP_FWD_NOGRAD, SWIGLU_OP_BWD = 0, 1, 2
STATUS = {0: "SWIGLU_OK", 1: "SWIGLU_ERR_INVALID_ARG", 2: "SWIGLU_ERR_ALIGNMENT",
          3: "SWIGLU_ERR_UNSUPPORTED", 4: "SWIGLU_ERR_WORKSPACE", 5: "SWIGLU_ERR_CUDA",
          6: "SWIGLU_ERR_DEVICE_TIMEOUT", 7: "SWIGLU_ERR_DEVICE_BOUNDS"}

_DT = {torch.bfloat16: SWIGLU_BF16, torch.float16: SWIGLU_F16, torch.float32: SWIGLU_F32_IEEE}

_lock = threading.Lock()
_lib = None
_loaded = {}  # path -> CDLL
_use_debug = False


class SwigluError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (%s)" % (where, STATUS.get(code, code), status_string(code)))


class W4Format(ctypes.Structure):
    """swiglu_mlp_w4_format: group size and zero-point flag of packed 4-bit experts."""
    _fields_ = [("group", ctypes.c_int), ("zeros", ctypes.c_int)]


class Options(ctypes.Structure):
    """swiglu_mlp_options: gate/down multipliers and weight-gradient accumulation."""
    _fields_ = [("gate_multiplier", ctypes.c_float), ("down_multiplier", ctypes.c_float),
                ("accumulate", ctypes.c_int)]


def _opts(gate_mul: float, down_mul: float, accumulate: bool):
    """NULL for the standard MLP, else a pointer to an Options."""
    if gate_mul == 1.0 and down_mul == 1.0 and not accumulate:
        return ctypes.c_void_p(0)
    return ctypes.byref(Options(float(gate_mul), float(down_mul), 1 if accumulate else 0))


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built): the release
    build, or the debug build while use_debug_library(True) is in effect."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _load(DEBUG_LIB_PATH if _use_debug else LIB_PATH)
        return _lib


def use_debug_library(on: bool) -> bool:
    """Routes every later call of this module to the debug build
    (libswiglu_mlp_debug.so: device index checks, SWIGLU_ERR_DEVICE_BOUNDS)
    or back to the release build; returns the previous setting.  Both stay
    loaded; each keeps its own process-wide settings (wait limit, SM-pair
    and few-token modes)."""
    global _lib, _use_debug
    with _lock:
        prev = _use_debug
        _use_debug = bool(on)
        _lib = None
    lib()
    return prev


def _load(path: str) -> ctypes.CDLL:
    if path in _loaded:
        return _loaded[path]
    if not os.path.exists(path):
        raise ImportError("%s is not built (run __graft_entry__.build() or python -m "
                          "backward_tcgen05_tma_gb300.build); no fallback exists"
                          % os.path.basename(path))
    L = ctypes.CDLL(path)
    vp, i64, ci, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.swiglu_mlp_element_bytes.restype = sz
    L.swiglu_mlp_element_bytes.argtypes = [ci]
    L.swiglu_mlp_saved_bytes.restype = sz
    L.swiglu_mlp_saved_bytes.argtypes = [i64, i64, ci]
    L.swiglu_mlp_workspace_bytes.restype = sz
    L.swiglu_mlp_workspace_bytes.argtypes = [i64, i64, i64, ci, ci]
    L.swiglu_mlp_workspace_min_bytes.restype = sz
    L.swiglu_mlp_workspace_min_bytes.argtypes = [i64, i64, i64, ci, ci]
    L.swiglu_mlp_fwd.restype = ci
    L.swiglu_mlp_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, sz, vp]
    L.swiglu_mlp_fwd_nograd.restype = ci
    L.swiglu_mlp_fwd_nograd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, sz, vp]
    L.swiglu_mlp_fwd_nograd_noalloc.restype = ci
    L.swiglu_mlp_fwd_nograd_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
    L.swiglu_mlp_graph_create_fwd_nograd.restype = ci
    L.swiglu_mlp_graph_create_fwd_nograd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp,
                                                     sz, ctypes.POINTER(vp)]
    L.swiglu_mlp_graph_launch.restype = ci
    L.swiglu_mlp_graph_launch.argtypes = [vp, vp]
    L.swiglu_mlp_graph_destroy.restype = ci
    L.swiglu_mlp_graph_destroy.argtypes = [vp]
    op = ctypes.c_void_p
    L.swiglu_mlp_fwd_ex.restype = ci
    L.swiglu_mlp_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, op, vp, sz, vp]
    L.swiglu_mlp_fwd_nograd_ex.restype = ci
    L.swiglu_mlp_fwd_nograd_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, op, vp, sz,
                                           vp]
    L.swiglu_mlp_bwd_ex.restype = ci
    L.swiglu_mlp_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, op, vp,
                                    sz, vp]
    L.swiglu_mlp_packed_weights_bytes.restype = sz
    L.swiglu_mlp_packed_weights_bytes.argtypes = [i64, i64, ci]
    L.swiglu_mlp_pack_weights.restype = ci
    L.swiglu_mlp_pack_weights.argtypes = [vp, vp, vp, i64, i64, ci, vp]
    L.swiglu_mlp_fwd_nograd_packed.restype = ci
    L.swiglu_mlp_fwd_nograd_packed.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, op, vp, sz, vp]
    L.swiglu_mlp_bwd.restype = ci
    L.swiglu_mlp_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, sz, vp]
    L.swiglu_mlp_query_error.restype = ci
    L.swiglu_mlp_query_error.argtypes = [vp, vp]
    L.swiglu_status_string.restype = ctypes.c_char_p
    L.swiglu_status_string.argtypes = [ci]
    L.swiglu_mlp_set_wait_limit_ns.restype = ctypes.c_uint64
    L.swiglu_mlp_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.swiglu_mlp_inject_stall_once.restype = None
    L.swiglu_mlp_inject_stall_once.argtypes = [ci]
    L.swiglu_mlp_last_launch_count.restype = ci
    L.swiglu_mlp_last_launch_count.argtypes = []
    fp = ctypes.c_void_p
    L.swiglu_mlp_test_elementwise.restype = ci
    L.swiglu_mlp_test_elementwise.argtypes = [ci, i64, fp, fp, vp, vp, vp, fp, vp, vp, vp, vp,
                                              ctypes.c_float, ctypes.c_float, vp]
    L.swiglu_mlp_set_cta_pairs.restype = ci
    L.swiglu_mlp_set_cta_pairs.argtypes = [ci]
    L.swiglu_mlp_set_nograd_fused.restype = ci
    L.swiglu_mlp_set_nograd_fused.argtypes = [ci]
    L.swiglu_mlp_set_wide_tiles.restype = ci
    L.swiglu_mlp_set_wide_tiles.argtypes = [ci]
    L.swiglu_mlp_profile_enable.restype = None
    L.swiglu_mlp_profile_enable.argtypes = [ci]
    L.swiglu_mlp_profile_read.restype = ci
    L.swiglu_mlp_profile_read.argtypes = [ci, vp, vp]
    L.swiglu_mlp_kernel_name.restype = ctypes.c_char_p
    L.swiglu_mlp_kernel_name.argtypes = [ci]
    L.swiglu_mlp_w4_packed_bytes.restype = sz
    L.swiglu_mlp_w4_packed_bytes.argtypes = [i64, i64, i64, ci, ci, ci]
    L.swiglu_mlp_w4_quantize.restype = ci
    L.swiglu_mlp_w4_quantize.argtypes = [vp, vp, vp, vp, i64, i64, ci, ci, vp]
    L.swiglu_mlp_w4_pack.restype = ci
    L.swiglu_mlp_w4_pack.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, vp]
    L.swiglu_mlp_w4_unpack.restype = ci
    L.swiglu_mlp_w4_unpack.argtypes = [vp, vp, i64, i64, i64, ci, ci, ci, ci, vp]
    L.swiglu_mlp_w4_workspace_bytes.restype = sz
    L.swiglu_mlp_w4_workspace_bytes.argtypes = [i64, i64, i64]
    L.swiglu_mlp_fwd_nograd_w4_workspace_bytes.restype = sz
    L.swiglu_mlp_fwd_nograd_w4_workspace_bytes.argtypes = [i64, i64, i64]
    L.swiglu_mlp_w4_linear.restype = ci
    L.swiglu_mlp_w4_linear.argtypes = [vp, vp, vp, i64, i64, i64, ci, ci, ci, vp, sz, vp]
    L.swiglu_mlp_fwd_nograd_w4.restype = ci
    L.swiglu_mlp_fwd_nograd_w4.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, op, vp,
                                           sz, vp]
    cf = ctypes.c_float
    L.swiglu_mlp_moe_workspace_bytes.restype = sz
    L.swiglu_mlp_moe_workspace_bytes.argtypes = [i64, i64, i64, i64, ci]
    L.swiglu_mlp_moe_route.restype = ci
    L.swiglu_mlp_moe_route.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, cf, ci, vp]
    L.swiglu_mlp_moe_experts.restype = ci
    L.swiglu_mlp_moe_experts.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, ci, vp, ci,
                                         op, vp, sz, vp]
    L.swiglu_mlp_moe_fwd_nograd.restype = ci
    L.swiglu_mlp_moe_fwd_nograd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, ci, ci,
                                            cf, vp, ci, op, vp, sz, vp]
    L.swiglu_mlp_debug_build.restype = ci
    L.swiglu_mlp_debug_build.argtypes = []
    L.swiglu_mlp_debug_narrow_once.restype = None
    L.swiglu_mlp_debug_narrow_once.argtypes = [ci]
    _loaded[path] = L
    return L


def declared_symbols() -> list[str]:
    """Function names declared in include/swiglu_mlp.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(swiglu_(?:mlp|status)_\w+)\s*\(", text)))


def status_string(code: int) -> str:
    return lib().swiglu_status_string(code).decode()


def dtype_code(dtype: torch.dtype) -> int:
    if dtype not in _DT:
        raise TypeError("unsupported dtype %s (bf16, fp16 or fp32)" % dtype)
    return _DT[dtype]


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _check(code: int, where: str):
    if code != 0:
        raise SwigluError(code, where)


def _device_check(ws, where: str):
    """While the debug build is in use: wait for the call and raise on the
    device status in its workspace (a failed index check, a timeout).  The
    release build returns at once, as every call is asynchronous."""
    if _use_debug:
        code = int(lib().swiglu_mlp_query_error(_ptr(ws), _stream(ws.device)))
        if code != 0:
            raise SwigluError(code, where + " (device)")


def workspace(M: int, D: int, H: int, dtype: torch.dtype, op: int, device,
              minimal: bool = False) -> torch.Tensor:
    """A zero-filled workspace: the recommended size, or with ``minimal`` the
    smallest accepted one (stream-K off where its partials would not fit)."""
    f = lib().swiglu_mlp_workspace_min_bytes if minimal else lib().swiglu_mlp_workspace_bytes
    n = f(M, D, H, dtype_code(dtype), op)
    return torch.zeros(int(n), dtype=torch.uint8, device=device)


def _dims(X, Wgu, Wd):
    M, D = X.shape
    H = Wgu.shape[0] // 2
    if Wgu.shape != (2 * H, D) or Wd.shape != (D, H):
        raise ValueError("shape mismatch: X %s, Wgu %s, Wd %s" % (tuple(X.shape), tuple(Wgu.shape),
                                                                   tuple(Wd.shape)))
    for t in (X, Wgu, Wd):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != X.dtype:
            raise ValueError("inputs must be contiguous CUDA tensors of one dtype")
    return M, D, H


def swiglu_mlp_fwd(X, Wgu, Wd, out: dict | None = None, ws=None, gate_mul: float = 1.0,
                   down_mul: float = 1.0):
    """Training forward: returns (Y [M,D], saved [M,3H]).  ``gate_mul`` /
    ``down_mul``: the multiplier variant (swiglu_mlp_fwd_ex)."""
    M, D, H = _dims(X, Wgu, Wd)
    out = out or {}
    Y = out.get("Y")
    Y = torch.empty(M, D, dtype=X.dtype, device=X.device) if Y is None else Y
    saved = out.get("saved")
    saved = torch.empty(M, 3 * H, dtype=X.dtype, device=X.device) if saved is None else saved
    ws = workspace(M, D, H, X.dtype, SWIGLU_OP_FWD, X.device) if ws is None else ws
    _check(lib().swiglu_mlp_fwd_ex(_ptr(X), _ptr(Wgu), _ptr(Wd), _ptr(Y), _ptr(saved), M, D, H,
                                   dtype_code(X.dtype), _opts(gate_mul, down_mul, False),
                                   _ptr(ws), ws.numel(), _stream(X.device)),
           "swiglu_mlp_fwd")
    _device_check(ws, "swiglu_mlp_fwd")
    return Y, saved


def swiglu_mlp_fwd_nograd(X, Wgu, Wd, out: dict | None = None, ws=None, gate_mul: float = 1.0,
                          down_mul: float = 1.0):
    """Inference forward: returns (Y [M,D], A [M,H]); G and U are never stored."""
    M, D, H = _dims(X, Wgu, Wd)
    out = out or {}
    Y = out.get("Y")
    Y = torch.empty(M, D, dtype=X.dtype, device=X.device) if Y is None else Y
    A = out.get("A")
    A = torch.empty(M, H, dtype=X.dtype, device=X.device) if A is None else A
    ws = workspace(M, D, H, X.dtype, SWIGLU_OP_FWD_NOGRAD, X.device) if ws is None else ws
    _check(lib().swiglu_mlp_fwd_nograd_ex(_ptr(X), _ptr(Wgu), _ptr(Wd), _ptr(Y), _ptr(A), M, D,
                                          H, dtype_code(X.dtype),
                                          _opts(gate_mul, down_mul, False), _ptr(ws), ws.numel(),
                                          _stream(X.device)),
           "swiglu_mlp_fwd_nograd")
    _device_check(ws, "swiglu_mlp_fwd_nograd")
    return Y, A


def swiglu_mlp_fwd_nograd_noalloc(X, Wgu, Wd, out: dict | None = None):
    """Few-token no-grad forward that allocates nothing in the library (its
    scratch is a static device array): returns (Y [M,D], A [M,H])."""
    M, D, H = _dims(X, Wgu, Wd)
    out = out or {}
    Y = out.get("Y")
    Y = torch.empty(M, D, dtype=X.dtype, device=X.device) if Y is None else Y
    A = out.get("A")
    A = torch.empty(M, H, dtype=X.dtype, device=X.device) if A is None else A
    _check(lib().swiglu_mlp_fwd_nograd_noalloc(_ptr(X), _ptr(Wgu), _ptr(Wd), _ptr(Y), _ptr(A), M,
                                               D, H, dtype_code(X.dtype), _stream(X.device)),
           "swiglu_mlp_fwd_nograd_noalloc")
    return Y, A


def swiglu_mlp_pack_weights(Wgu, Wd, packed=None) -> torch.Tensor:
    """The packed copy of (Wgu [2H,D], Wd [D,H]) that
    swiglu_mlp_fwd_nograd_packed streams (a uint8 device tensor)."""
    H2, D = Wgu.shape
    H = H2 // 2
    if Wgu.shape != (2 * H, D) or Wd.shape != (D, H):
        raise ValueError("expected Wgu [2H, D] and Wd [D, H]")
    n = int(lib().swiglu_mlp_packed_weights_bytes(D, H, dtype_code(Wgu.dtype)))
    if n == 0:
        raise SwigluError(3, "swiglu_mlp_pack_weights")
    packed = torch.empty(n, dtype=torch.uint8, device=Wgu.device) if packed is None else packed
    if packed.numel() < n:
        raise ValueError("packed buffer too small")
    _check(lib().swiglu_mlp_pack_weights(_ptr(Wgu), _ptr(Wd), _ptr(packed), D, H,
                                         dtype_code(Wgu.dtype), _stream(Wgu.device)),
           "swiglu_mlp_pack_weights")
    return packed


def swiglu_mlp_fwd_nograd_packed(X, packed, H: int, out: dict | None = None, ws=None,
                                 gate_mul: float = 1.0, down_mul: float = 1.0):
    """Few-token (M <= 64) no-grad forward on weights packed by
    swiglu_mlp_pack_weights: returns (Y [M,D], A [M,H])."""
    M, D = X.shape
    out = out or {}
    Y = out.get("Y")
    Y = torch.empty(M, D, dtype=X.dtype, device=X.device) if Y is None else Y
    A = out.get("A")
    A = torch.empty(M, H, dtype=X.dtype, device=X.device) if A is None else A
    ws = workspace(M, D, H, X.dtype, SWIGLU_OP_FWD_NOGRAD, X.device) if ws is None else ws
    _check(lib().swiglu_mlp_fwd_nograd_packed(_ptr(X), _ptr(packed), _ptr(Y), _ptr(A), M, D, H,
                                              dtype_code(X.dtype),
                                              _opts(gate_mul, down_mul, False), _ptr(ws),
                                              ws.numel(), _stream(X.device)),
           "swiglu_mlp_fwd_nograd_packed")
    _device_check(ws, "swiglu_mlp_fwd_nograd_packed")
    return Y, A


class FwdNogradGraph:
    """A no-grad forward recorded once as a CUDA graph (swiglu_mlp_graph_*)
    on static buffers ``X`` [M,D], ``Y`` [M,D], ``A`` [M,H] and a workspace;
    each call copies new tokens into ``X`` (unless they are ``X`` itself),
    replays the graph on the current stream and returns ``Y``.  Holds
    references to every buffer the graph reads or writes."""

    def __init__(self, Wgu, Wd, M: int, X=None, out: dict | None = None, ws=None):
        D = Wd.shape[0]
        dev, dt = Wgu.device, Wgu.dtype
        self.X = torch.empty(M, D, dtype=dt, device=dev) if X is None else X
        M, D, H = _dims(self.X, Wgu, Wd)
        out = out or {}
        self.Y = out.get("Y")
        self.Y = torch.empty(M, D, dtype=dt, device=dev) if self.Y is None else self.Y
        self.A = out.get("A")
        self.A = torch.empty(M, H, dtype=dt, device=dev) if self.A is None else self.A
        self.ws = workspace(M, D, H, dt, SWIGLU_OP_FWD_NOGRAD, dev) if ws is None else ws
        self.Wgu, self.Wd = Wgu, Wd
        torch.cuda.synchronize(dev)  # the workspace's zero-fill is complete before any replay
        h = ctypes.c_void_p(0)
        L = lib()
        with torch.cuda.device(dev):
            _check(L.swiglu_mlp_graph_create_fwd_nograd(
                _ptr(self.X), _ptr(Wgu), _ptr(Wd), _ptr(self.Y), _ptr(self.A), M, D, H,
                dtype_code(dt), _ptr(self.ws), self.ws.numel(), ctypes.byref(h)),
                "swiglu_mlp_graph_create_fwd_nograd")
        self._h = h
        self._L = L

    def launch(self, stream=None):
        s = torch.cuda.current_stream(self.X.device) if stream is None else stream
        _check(self._L.swiglu_mlp_graph_launch(self._h, ctypes.c_void_p(s.cuda_stream)),
               "swiglu_mlp_graph_launch")
        if _use_debug:  # as _device_check, with the graph's own library
            code = int(self._L.swiglu_mlp_query_error(_ptr(self.ws),
                                                      ctypes.c_void_p(s.cuda_stream)))
            if code != 0:
                raise SwigluError(code, "swiglu_mlp_graph_launch (device)")

    def __call__(self, x=None):
        if x is not None and x.data_ptr() != self.X.data_ptr():
            self.X.copy_(x)
        self.launch()
        return self.Y

    def close(self):
        """Destroys the graph after pending launches on this device finish
        (so the buffers it holds may be freed afterwards)."""
        if getattr(self, "_h", None) is not None and self._h.value:
            torch.cuda.synchronize(self.X.device)
            _check(self._L.swiglu_mlp_graph_destroy(self._h), "swiglu_mlp_graph_destroy")
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def swiglu_mlp_bwd(dY, X, Wgu, Wd, saved, out: dict | None = None, ws=None,
                   gate_mul: float = 1.0, down_mul: float = 1.0, accumulate: bool = False):
    """Backward: returns (dX [M,D], dWgu [2H,D], dWd [D,H]).  Overwrites the
    G/U columns of ``saved`` with dG/dU (a second call on it is undefined).
    ``accumulate``: add into the dWgu / dWd given in ``out`` (beta = 1)."""
    M, D, H = _dims(X, Wgu, Wd)
    if dY.shape != (M, D) or saved.shape != (M, 3 * H):
        raise ValueError("dY/saved shape mismatch")
    out = out or {}
    dX = out.get("dX")
    dX = torch.empty(M, D, dtype=X.dtype, device=X.device) if dX is None else dX
    dWgu = out.get("dWgu")
    dWgu = torch.empty(2 * H, D, dtype=X.dtype, device=X.device) if dWgu is None else dWgu
    dWd = out.get("dWd")
    dWd = torch.empty(D, H, dtype=X.dtype, device=X.device) if dWd is None else dWd
    ws = workspace(M, D, H, X.dtype, SWIGLU_OP_BWD, X.device) if ws is None else ws
    if accumulate and (out.get("dWgu") is None or out.get("dWd") is None):
        raise ValueError("accumulate needs the held dWgu and dWd in out")
    _check(lib().swiglu_mlp_bwd_ex(_ptr(dY), _ptr(X), _ptr(Wgu), _ptr(Wd), _ptr(saved),
                                   _ptr(dX), _ptr(dWgu), _ptr(dWd), M, D, H,
                                   dtype_code(X.dtype), _opts(gate_mul, down_mul, accumulate),
                                   _ptr(ws), ws.numel(), _stream(X.device)),
           "swiglu_mlp_bwd")
    _device_check(ws, "swiglu_mlp_bwd")
    return dX, dWgu, dWd


# The few-token calls below last a few microseconds, so their Python part is
# kept short: plain integers for pointers and streams, no temporaries.  (A torch
# without CUDA lacks this function, and has no tensors that would need it.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _serving_checks(X, *others) -> int:
    """Contiguous CUDA tensors of X's device; returns X's current stream."""
    dev = X.get_device()
    ok = dev >= 0 and X.is_contiguous()
    for t in others:
        ok = ok and t.get_device() == dev and t.is_contiguous()
    if not ok:
        raise ValueError("inputs and outputs must be contiguous CUDA tensors of one device")
    return _raw_stream(dev)


def _out(out, name, shape, dtype, device):
    """The caller's output tensor, checked, or a new one."""
    t = out.get(name) if out else None
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("out[%r] must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, tuple(shape), device))
    return t


def _ws(ws, size, device):
    """The caller's workspace (its size is checked by the call) or a new one."""
    return torch.zeros(int(size()), dtype=torch.uint8, device=device) if ws is None else ws


class W4Weights:
    """One 4-bit matrix [N, K], or ``experts`` of them, in the layout the
    few-token products stream (swiglu_mlp_w4_pack).  ``gate_up``: the rows are
    a [Wg; Wu] pair."""

    def __init__(self, packed, N, K, group, zeros, gate_up, dtype, experts=None):
        self.packed, self.N, self.K, self.group = packed, int(N), int(K), int(group)
        self.zeros, self.gate_up, self.dtype = bool(zeros), bool(gate_up), dtype
        self.experts = experts
        self.shape = (self.N, self.K) if experts is None else (experts, self.N, self.K)
        self.format = W4Format(self.group, int(self.zeros))

    @property
    def device(self):
        return self.packed.device

    def __repr__(self):
        return "W4Weights(%s, group=%d, zeros=%s, gate_up=%s, dtype=%s)" % (
            tuple(self.shape), self.group, self.zeros, self.gate_up, self.dtype)


def swiglu_mlp_w4_quantize(W, group: int = 128, zeros: bool = False):
    """Rounds W [N, K] or [E, N, K] to 4 bits: (codes uint8 [.., N, K/2],
    scales [.., N, ceil(K/group)] in W's type, zero points uint8 or None)."""
    st = _serving_checks(W)
    if W.dim() not in (2, 3):
        raise ValueError("expected W [N, K] or [E, N, K], got %s" % (tuple(W.shape),))
    *lead, N, K = W.shape
    rows = W.numel() // K if K else 0
    if group not in (32, 64, 128):
        raise SwigluError(1, "swiglu_mlp_w4_quantize")
    ng = -(-K // group)
    codes = torch.empty(*lead, N, K // 2, dtype=torch.uint8, device=W.device)
    scales = torch.empty(*lead, N, ng, dtype=W.dtype, device=W.device)
    zp = torch.empty(*lead, N, ng, dtype=torch.uint8, device=W.device) if zeros else None
    _check(lib().swiglu_mlp_w4_quantize(_ptr(W), _ptr(codes), _ptr(scales), _ptr(zp), rows, K,
                                        group, dtype_code(W.dtype), st),
           "swiglu_mlp_w4_quantize")
    return codes, scales, zp


def swiglu_mlp_w4_pack(codes, scales, zeros=None, group: int = 128,
                       gate_up: bool = False) -> W4Weights:
    """The packed copy of 4-bit weights (codes uint8 [.., N, K/2], scales
    [.., N, ceil(K/group)] in the activations' type, optional zero points) that
    the few-token products stream.  Zero points are whole numbers of 0..15, and
    others are refused (one wait for the device where there are zero points);
    formats that hold a zero point of 16 have no such copy."""
    st = _serving_checks(codes, scales, *(() if zeros is None else (zeros,)))
    if codes.dim() not in (2, 3) or codes.dtype != torch.uint8:
        raise ValueError("expected uint8 codes [N, K/2] or [E, N, K/2]")
    *lead, N, half = codes.shape
    E, K = (lead[0] if lead else 1), 2 * half
    want = (*lead, N, -(-K // group))
    if tuple(scales.shape) != want:
        raise ValueError("expected scales of shape %s, got %s" % (want, tuple(scales.shape)))
    if zeros is not None and (tuple(zeros.shape) != want or zeros.dtype != torch.uint8):
        raise ValueError("expected uint8 zero points of shape %s" % (want,))
    if zeros is not None and zeros.numel() and int(zeros.max()) > 15:
        raise ValueError("zero points must be 0..15, got %d" % int(zeros.max()))
    zp = zeros is not None
    n = int(lib().swiglu_mlp_w4_packed_bytes(E, N, K, group, int(zp), int(gate_up)))
    packed = torch.empty(n, dtype=torch.uint8, device=codes.device)
    _check(lib().swiglu_mlp_w4_pack(_ptr(codes), _ptr(scales), _ptr(zeros), _ptr(packed), E, N, K,
                                    group, int(gate_up), dtype_code(scales.dtype), st),
           "swiglu_mlp_w4_pack")
    return W4Weights(packed, N, K, group, zp, gate_up, scales.dtype, lead[0] if lead else None)


def swiglu_mlp_w4_unpack(W: W4Weights) -> torch.Tensor:
    """The 16-bit weights a packed copy stands for ([N, K] or [E, N, K])."""
    out = torch.empty(W.shape, dtype=W.dtype, device=W.device)
    _check(lib().swiglu_mlp_w4_unpack(_ptr(W.packed), _ptr(out), W.experts or 1, W.N, W.K, W.group,
                                      int(W.zeros), int(W.gate_up), dtype_code(W.dtype),
                                      ctypes.c_void_p(_stream(W.device))),
           "swiglu_mlp_w4_unpack")
    return out


def w4_linear_workspace(M: int, N: int, K: int, device) -> torch.Tensor:
    """A zero-filled workspace for swiglu_mlp_w4_linear."""
    return _ws(None, lambda: lib().swiglu_mlp_w4_workspace_bytes(M, N, K), device)


def w4_workspace(M: int, D: int, H: int, device) -> torch.Tensor:
    """A zero-filled workspace for swiglu_mlp_fwd_nograd_w4."""
    return _ws(None, lambda: lib().swiglu_mlp_fwd_nograd_w4_workspace_bytes(M, D, H), device)


def moe_workspace(T: int, D: int, H: int, E: int, top_k: int, device) -> torch.Tensor:
    """A zero-filled workspace for swiglu_mlp_moe_experts / _moe_fwd_nograd."""
    return _ws(None, lambda: lib().swiglu_mlp_moe_workspace_bytes(T, D, H, E, top_k), device)


def _w4_match(X, K, *weights):
    for W in weights:
        if W.dtype != X.dtype:
            raise ValueError("4-bit weights for %s, activations %s" % (W.dtype, X.dtype))
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError("expected X [M, %d], got %s" % (K, tuple(X.shape)))


def swiglu_mlp_w4_linear(X, W: W4Weights, out: dict | None = None, ws=None):
    """Y [M, N] = X [M, K] W^T for up to 64 tokens and 4-bit weights."""
    if W.gate_up or W.experts is not None:
        raise ValueError("expected one matrix packed without gate_up")
    _w4_match(X, W.K, W)
    M = X.shape[0]
    Y = _out(out, "Y", (M, W.N), X.dtype, X.device)
    L = _lib or lib()
    ws = _ws(ws, lambda: L.swiglu_mlp_w4_workspace_bytes(M, W.N, W.K), X.device)
    st = _serving_checks(X, W.packed, ws)
    _check(L.swiglu_mlp_w4_linear(X.data_ptr(), W.packed.data_ptr(), Y.data_ptr(), M, W.N, W.K,
                                  W.group, W.zeros, dtype_code(X.dtype), ws.data_ptr(), ws.numel(),
                                  st),
           "swiglu_mlp_w4_linear")
    _device_check(ws, "swiglu_mlp_w4_linear")
    return Y


def swiglu_mlp_fwd_nograd_w4(X, Wgu: W4Weights, Wd: W4Weights, out: dict | None = None, ws=None,
                             gate_mul: float = 1.0, down_mul: float = 1.0):
    """The no-grad MLP on 4-bit weights for up to 64 tokens: (Y [M,D], A [M,H])."""
    if not Wgu.gate_up or Wd.gate_up or Wgu.experts is not None or Wd.experts is not None:
        raise ValueError("expected Wgu packed with gate_up and Wd without")
    H, D = Wd.K, Wd.N
    if Wgu.shape != (2 * H, D) or Wgu.group != Wd.group or Wgu.zeros != Wd.zeros:
        raise ValueError("mismatch: Wgu %r, Wd %r" % (Wgu, Wd))
    _w4_match(X, D, Wgu, Wd)
    M = X.shape[0]
    Y = _out(out, "Y", (M, D), X.dtype, X.device)
    A = _out(out, "A", (M, H), X.dtype, X.device)
    L = _lib or lib()
    ws = _ws(ws, lambda: L.swiglu_mlp_fwd_nograd_w4_workspace_bytes(M, D, H), X.device)
    st = _serving_checks(X, Wgu.packed, Wd.packed, ws)
    _check(L.swiglu_mlp_fwd_nograd_w4(X.data_ptr(), Wgu.packed.data_ptr(), Wd.packed.data_ptr(),
                                      Y.data_ptr(), A.data_ptr(), M, D, H, Wd.group, Wd.zeros,
                                      dtype_code(X.dtype), _opts(gate_mul, down_mul, False),
                                      ws.data_ptr(), ws.numel(), st),
           "swiglu_mlp_fwd_nograd_w4")
    _device_check(ws, "swiglu_mlp_fwd_nograd_w4")
    return Y, A


def swiglu_mlp_moe_route(X, Wr, top_k: int, norm_topk: bool = True, route_scale: float = 1.0,
                         out: dict | None = None):
    """The router: (idx int32 [T, top_k], weights fp32 [T, top_k])."""
    T, D = X.shape
    E = Wr.shape[0]
    if Wr.shape != (E, D) or Wr.dtype != X.dtype:
        raise ValueError("expected Wr [E, %d] of %s, got %s %s" % (D, X.dtype, tuple(Wr.shape),
                                                                   Wr.dtype))
    idx = _out(out, "idx", (T, top_k), torch.int32, X.device)
    w = _out(out, "weights", (T, top_k), torch.float32, X.device)
    st = _serving_checks(X, Wr)
    _check(lib().swiglu_mlp_moe_route(X.data_ptr(), Wr.data_ptr(), idx.data_ptr(), w.data_ptr(), T,
                                      D, E, top_k, int(norm_topk), float(route_scale),
                                      dtype_code(X.dtype), st),
           "swiglu_mlp_moe_route")
    return idx, w


def _experts(X, Wgu, Wd):
    """(T, D, H, E, the format struct or None, the two buffers) of a layer."""
    w4 = isinstance(Wgu, W4Weights)
    if X.dim() != 2 or w4 != isinstance(Wd, W4Weights) or len(Wd.shape) != 3:
        raise ValueError("expected X [T, D], and Wgu [E, 2H, D] and Wd [E, D, H] either as 16-bit "
                         "tensors or as W4Weights")
    T, D = X.shape
    E, H = Wd.shape[0], Wd.shape[2]
    if Wgu.shape != (E, 2 * H, D) or Wd.shape != (E, D, H):
        raise ValueError("expected Wgu [E, 2H, %d] and Wd [E, %d, H], got %s and %s"
                         % (D, D, tuple(Wgu.shape), tuple(Wd.shape)))
    if Wgu.dtype != X.dtype or Wd.dtype != X.dtype:
        raise ValueError("activations and experts must have one dtype")
    if not w4:
        return T, D, H, E, None, Wgu, Wd
    if not Wgu.gate_up or Wd.gate_up or Wgu.group != Wd.group or Wgu.zeros != Wd.zeros:
        raise ValueError("mismatch: Wgu %r, Wd %r" % (Wgu, Wd))
    return T, D, H, E, ctypes.byref(Wd.format), Wgu.packed, Wd.packed


def swiglu_mlp_moe_experts(X, idx, weights, Wgu, Wd, out: dict | None = None, ws=None,
                           gate_mul: float = 1.0, down_mul: float = 1.0):
    """Y[t] = sum_j weights[t, j] MLP_{idx[t, j]}(X[t]) for up to 64 tokens:
    Y [T, D].  Wgu [E, 2H, D] and Wd [E, D, H], or their W4Weights.  An idx
    outside 0..E-1 is no expert."""
    T, D, H, E, fmt, gu, down = _experts(X, Wgu, Wd)
    if idx.dim() != 2 or idx.shape[0] != T or idx.dtype != torch.int32 \
            or weights.shape != idx.shape or weights.dtype != torch.float32:
        raise ValueError("expected idx int32 [T, top_k] and weights fp32 of its shape")
    k = idx.shape[1]
    Y = _out(out, "Y", (T, D), X.dtype, X.device)
    L = _lib or lib()
    ws = _ws(ws, lambda: L.swiglu_mlp_moe_workspace_bytes(T, D, H, E, k), X.device)
    st = _serving_checks(X, idx, weights, gu, down, ws)
    _check(L.swiglu_mlp_moe_experts(X.data_ptr(), idx.data_ptr(), weights.data_ptr(), gu.data_ptr(),
                                    down.data_ptr(), Y.data_ptr(), T, D, H, E, k, fmt,
                                    dtype_code(X.dtype), _opts(gate_mul, down_mul, False),
                                    ws.data_ptr(), ws.numel(), st),
           "swiglu_mlp_moe_experts")
    _device_check(ws, "swiglu_mlp_moe_experts")
    return Y


def swiglu_mlp_moe_fwd_nograd(X, Wr, Wgu, Wd, top_k: int, norm_topk: bool = True,
                              route_scale: float = 1.0, out: dict | None = None, ws=None,
                              gate_mul: float = 1.0, down_mul: float = 1.0):
    """A mixture-of-experts layer for up to 64 tokens, without gradients:
    (Y [T, D], idx int32 [T, top_k], weights fp32 [T, top_k])."""
    T, D, H, E, fmt, gu, down = _experts(X, Wgu, Wd)
    if Wr.shape != (E, D) or Wr.dtype != X.dtype:
        raise ValueError("expected Wr [%d, %d] of %s, got %s %s" % (E, D, X.dtype, tuple(Wr.shape),
                                                                    Wr.dtype))
    Y = _out(out, "Y", (T, D), X.dtype, X.device)
    idx = _out(out, "idx", (T, top_k), torch.int32, X.device)
    w = _out(out, "weights", (T, top_k), torch.float32, X.device)
    L = _lib or lib()
    ws = _ws(ws, lambda: L.swiglu_mlp_moe_workspace_bytes(T, D, H, E, top_k), X.device)
    st = _serving_checks(X, Wr, gu, down, ws)
    _check(L.swiglu_mlp_moe_fwd_nograd(X.data_ptr(), Wr.data_ptr(), gu.data_ptr(), down.data_ptr(),
                                       Y.data_ptr(), idx.data_ptr(), w.data_ptr(), T, D, H, E,
                                       top_k, int(norm_topk), float(route_scale), fmt,
                                       dtype_code(X.dtype), _opts(gate_mul, down_mul, False),
                                       ws.data_ptr(), ws.numel(), st),
           "swiglu_mlp_moe_fwd_nograd")
    _device_check(ws, "swiglu_mlp_moe_fwd_nograd")
    return Y, idx, w


def swiglu_mlp_query_error(ws) -> int:
    """Synchronises the current stream and returns the device error status."""
    return int(lib().swiglu_mlp_query_error(_ptr(ws), _stream(ws.device)))


def swiglu_mlp_set_wait_limit_ns(ns: int) -> int:
    return int(lib().swiglu_mlp_set_wait_limit_ns(int(ns)))


def swiglu_mlp_inject_stall_once(on: bool | int = True) -> None:
    """True / 1: stall the next tensor-core launch; n: the n-th from now;
    False / 0: clear."""
    lib().swiglu_mlp_inject_stall_once(int(on))


def swiglu_mlp_last_launch_count() -> int:
    return int(lib().swiglu_mlp_last_launch_count())


def swiglu_mlp_set_cta_pairs(mode: int = 1) -> int:
    """Tensor-core GEMMs on SM pairs: 1 = by size (default), 2 = always,
    0 = never; returns the previous mode."""
    return int(lib().swiglu_mlp_set_cta_pairs(int(mode)))


def swiglu_mlp_set_wide_tiles(mode: int = 1) -> int:
    """Weight-gradient and dX GEMMs on SM pairs: 1 = 512-column tiles by
    size (the default), 0 = 256-column tiles, 2 = 512-column tiles always;
    returns the previous mode."""
    return int(lib().swiglu_mlp_set_wide_tiles(int(mode)))


def swiglu_mlp_set_nograd_fused(mode: int = 0) -> int:
    """Few-token no-grad calls: 0 two kernels (the default), 1 the fused kernel
    for 33..64 tokens, 2 always the fused kernel; returns the previous mode."""
    return int(lib().swiglu_mlp_set_nograd_fused(int(mode)))


def swiglu_mlp_profile_enable(on: bool = True) -> None:
    lib().swiglu_mlp_profile_enable(1 if on else 0)


def swiglu_mlp_profile_read() -> dict:
    """{kernel name: (launches, total device ms)} since the previous read."""
    n = 64
    launches = (ctypes.c_int64 * n)()
    ms = (ctypes.c_double * n)()
    k = lib().swiglu_mlp_profile_read(n, ctypes.cast(launches, ctypes.c_void_p),
                                      ctypes.cast(ms, ctypes.c_void_p))
    if k < 0:
        raise SwigluError(5, "swiglu_mlp_profile_read")
    out = {}
    for i in range(k):
        if launches[i]:
            out[lib().swiglu_mlp_kernel_name(i).decode()] = (int(launches[i]), float(ms[i]))
    return out


def swiglu_mlp_test_elementwise(dtype: torch.dtype, acc_g=None, acc_u=None, dA=None, gs=None,
                                us=None, gate_mul: float = 1.0, down_mul: float = 1.0) -> dict:
    """Test hook: the tensor-core epilogues' elementwise stage applied to the
    given values (1-D CUDA tensors, length a multiple of 32).  Forward from
    fp32 accumulators acc_g, acc_u -> {"A", "G", "U"}; backward from the fp32
    dA and the stored gs, us (``dtype``) -> {"dG", "dU"}."""
    fwd, bwd = acc_g is not None, dA is not None
    ref = acc_g if fwd else dA
    n = ref.numel()
    out = {}
    new = lambda: torch.empty(n, dtype=dtype, device=ref.device)
    if fwd:
        out = {"A": new(), "G": new(), "U": new()}
    if bwd:
        out.update({"dG": new(), "dU": new()})
    _check(lib().swiglu_mlp_test_elementwise(
        dtype_code(dtype), n, _ptr(acc_g), _ptr(acc_u), _ptr(out.get("A")), _ptr(out.get("G")),
        _ptr(out.get("U")), _ptr(dA), _ptr(gs), _ptr(us), _ptr(out.get("dG")),
        _ptr(out.get("dU")), float(gate_mul), float(down_mul), _stream(ref.device)),
        "swiglu_mlp_test_elementwise")
    return out
