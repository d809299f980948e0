"""AWQ W4A16 group-quantized linear layer for NVIDIA B200 (sm_100a).

A thin ctypes binding over ``libawq_b200.so`` (C ABI in ``include/awq_b200.h``).
This module only marshals arguments: PyTorch provides device memory and the
current CUDA stream; every step of the computation runs in the library's
kernels.  There is no fallback: if the shared library is missing or the device
is not sm_100, the calls raise.

Every tensor argument is checked here (type, dtype, shape, device,
contiguity) before the C ABI is called: the library sees raw device pointers
and cannot tell a mis-shaped tensor from a correct one.

Functions (names follow the C ABI):
  act_stats(xcal)                  -> m float32 [K]
  compute_scales(m)                -> s float16 [K]
  quantize_pack(W, s)              -> (Q int32 [K/8,N], scales float16 [K/128,N], zeros int32 [K/128,N/8])
  quantize_pack(W, s, zero_point=False) -> (Q, scales, None)   symmetric grid, zero point 8
  quantize_pack_clip(W, s, xcal)   -> (Q, scales, zeros, ratio_index): with weight clipping
  fold_inverse_scale(a, s)         -> fp16(a / s), a [K] or [rows,K] (1/s folded upstream)
  w4a16_gemv(X, s, Q, scales, zeros)   X [1,K] -> Y [1,N]   (zeros None: symmetric weights;
                                                             s None: X already holds X/s)
  w4a16_gemm(X, s, Q, scales, zeros)   X [M,K] -> Y [M,N]
  scales_alpha(m, j)               -> s float16 [K] of grid point alpha = j/8
  scale_search(xcal, W)            -> (s_best float16 [K], j_best, losses float64 [9]): the scale
                                      s = m^(j/8) (normalised) whose quantized layer has the
                                      smallest output error on the calibration rows
  QuantLinear(Q, scales, zeros, s)     a quantized layer ("WQLinear"): weights checked once,
                                       layer(X) -> Y with only X and Y checked per call
  w4a16_gemm_epilogue(X, s, Q, scales, zeros, bias, act, gated, residual)
                                       the product with bias, activation, gate and residual
                                       before its rounding (QuantLinear takes the same)
  interleave_gate_up(gate, up)         weight columns as a gated product wants them
  KV4Pages, KV4Cache                   a paged key/value cache in 4 bits: pages and slots of a
                                       step from request lengths, store, load, attention
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libawq_b200.so")

GROUP_SIZE = 128
W_BIT = 4
MAX_CALIB_ROWS = 8192
ABI_VERSION = 5

STATUS = {
    0: "AWQ_OK", 1: "AWQ_ERR_NULL", 2: "AWQ_ERR_SHAPE", 3: "AWQ_ERR_ALIGN",
    4: "AWQ_ERR_NONFINITE", 5: "AWQ_ERR_ARCH", 6: "AWQ_ERR_CUDA",
    7: "AWQ_ERR_DEVICE_TIMEOUT", 8: "AWQ_ERR_WORKSPACE", 9: "AWQ_ERR_RANGE", 10: "AWQ_ERR_CAPACITY",
}
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_NONFINITE, ERR_ARCH, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(9)
ERR_RANGE, ERR_CAPACITY = 9, 10

# activations of a fused epilogue (awq_act_t)
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
KV4_MAX_REQUESTS = 4096

# exported symbols, in declaration order of include/awq_b200.h
SYMBOLS = (
    "awq_status_string", "awq_abi_version", "awq_act_stats", "awq_compute_scales",
    "awq_quantize_pack", "awq_quantize_pack_symmetric", "awq_quantize_pack_clip",
    "awq_fold_inverse_scale",
    "awq_w4a16_gemv_workspace_size",
    "awq_w4a16_gemv",
    "awq_w4a16_gemm_workspace_size", "awq_w4a16_gemm",
    "awq_scales_alpha", "awq_scale_search_workspace_size", "awq_scale_search",
    "awq_w4a16_gemm_noalloc",
    "awq_w4a16_gemm_epilogue",
    "awq_kv4_page_bytes", "awq_kv4_reserve", "awq_kv4_release", "awq_kv4_append", "awq_kv4_load",
    "awq_kv4_attention_workspace_size", "awq_kv4_attention",
)
NOALLOC_SCRATCH_BYTES = 24 << 20


class AwqError(RuntimeError):
    def __init__(self, code: int, where: str):
        name = STATUS.get(code, f"status {code}")
        super().__init__(f"{where}: {name}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libawq_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m weight_only_quantization_quantize_b200._build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.awq_status_string.argtypes = [ctypes.c_int]
        L.awq_status_string.restype = ctypes.c_char_p
        L.awq_abi_version.argtypes = []
        L.awq_abi_version.restype = ctypes.c_int
        L.awq_act_stats.argtypes = [P, I64, I64, P, P, P]
        L.awq_compute_scales.argtypes = [P, I64, P, P, P]
        L.awq_quantize_pack.argtypes = [P, P, I64, I64, P, P, P, P, P]
        L.awq_quantize_pack_symmetric.argtypes = [P, P, I64, I64, P, P, P, P]
        L.awq_fold_inverse_scale.argtypes = [P, I64, I64, P, P, P, P]
        L.awq_quantize_pack_clip.argtypes = [P, P, P, I64, I64, I64, ctypes.c_int32, P, P, P, P, P, P]
        L.awq_w4a16_gemv_workspace_size.argtypes = [I64, I64]
        L.awq_w4a16_gemv_workspace_size.restype = SZ
        L.awq_w4a16_gemv.argtypes = [P, P, P, P, P, I64, I64, P, P, SZ, P, P]
        L.awq_w4a16_gemm_workspace_size.argtypes = [I64, I64, I64]
        L.awq_w4a16_gemm_workspace_size.restype = SZ
        L.awq_w4a16_gemm.argtypes = [P, P, P, P, P, I64, I64, I64, P, P, SZ, P, P]
        L.awq_w4a16_gemm_noalloc.argtypes = [P, P, P, P, P, I64, I64, I64, P, P, P]
        L.awq_scales_alpha.argtypes = [P, I64, ctypes.c_int32, P, P, P]
        L.awq_scale_search_workspace_size.argtypes = [I64, I64, I64]
        L.awq_scale_search_workspace_size.restype = SZ
        L.awq_scale_search.argtypes = [P, I64, I64, P, I64, P, P, P, P, SZ, P, P]
        I32, F32 = ctypes.c_int32, ctypes.c_float
        L.awq_w4a16_gemm_epilogue.argtypes = [P, P, P, P, P, I64, I64, I64, P, I32, I32, P, P, P, SZ, P, P]
        L.awq_kv4_page_bytes.argtypes = [I64, I64]
        L.awq_kv4_page_bytes.restype = SZ
        L.awq_kv4_reserve.argtypes = [P, P, I64, I64, P, I64, P, P, I64, I64, P, P, P, P, P, P, P]
        L.awq_kv4_release.argtypes = [P, P, I64, I64, P, I64, P, P, I64, P, P]
        L.awq_kv4_append.argtypes = [P, I64, P, I64, P, I64, I64, I64, P, I64, I64, P, P]
        L.awq_kv4_load.argtypes = [P, I64, I64, I64, P, I64, I64, P, P, P, P]
        L.awq_kv4_attention_workspace_size.argtypes = [I64]
        L.awq_kv4_attention_workspace_size.restype = SZ
        L.awq_kv4_attention.argtypes = [P, I64, I64, I64, P, I64, I64, I64, I64, P, I64, P, P, I64, I64, F32, I64,
                                        P, P, SZ, P, P]
        for name in ("awq_w4a16_gemm_epilogue", "awq_kv4_reserve", "awq_kv4_release", "awq_kv4_append",
                     "awq_kv4_load", "awq_kv4_attention"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("awq_act_stats", "awq_compute_scales", "awq_quantize_pack",
                     "awq_quantize_pack_symmetric", "awq_quantize_pack_clip", "awq_fold_inverse_scale",
                     "awq_w4a16_gemv",
                     "awq_w4a16_gemm", "awq_scales_alpha", "awq_scale_search",
                     "awq_w4a16_gemm_noalloc"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().awq_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(dev: torch.device) -> int:
    """The current CUDA stream of `dev` as a raw cudaStream_t value."""
    return torch._C._cuda_getCurrentRawStream(dev.index if dev.index is not None
                                              else torch.cuda.current_device())


def _stream(t: torch.Tensor):
    return _raw_stream(t.device)


def _on(dev: torch.device):
    """The device context for a call: a no-op when `dev` is already current."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _need(t, dtype, shape, name, device=None):
    """Check a tensor argument: CUDA, dtype, exact shape (None = any extent),
    contiguous, and on `device` when given."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if isinstance(shape, int):
        if t.dim() != shape:
            raise ValueError(f"{name} must have {shape} dims, got {tuple(t.shape)}")
    else:
        if t.dim() != len(shape) or any(e is not None and e != d for e, d in zip(shape, t.shape)):
            want = tuple("*" if e is None else e for e in shape)
            raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _check(code: int, where: str):
    if code != OK:
        raise AwqError(code, where)


_current_device = torch._C._cuda_getDevice
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _call(dev: torch.device, where: str, fn, *args):
    """One C call on `dev`, which costs a device switch only when another one is current."""
    if dev.index == _current_device():
        code = fn(*args)
    else:
        with torch.cuda.device(dev):
            code = fn(*args)
    if code != OK:
        raise AwqError(code, where)


def new_status(device) -> torch.Tensor:
    """A zeroed device status word for the calls' dev_status argument."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def raise_on_status(status: torch.Tensor, where: str = "device"):
    """Synchronize on the status word and raise if a kernel recorded an error."""
    code = int(status.item())
    if code != OK:
        raise AwqError(code, where)


def _need_status(status, device):
    if status is not None:
        _need(status, torch.int32, (None,), "status", device)
        if status.numel() < 1:
            raise ValueError("status must hold at least one int32")


def act_stats(xcal: torch.Tensor, status: torch.Tensor | None = None) -> torch.Tensor:
    """m[k] = mean_r |xcal[r,k]| (exact), float32 [K]."""
    _need(xcal, torch.float16, 2, "xcal")
    _need_status(status, xcal.device)
    R, K = xcal.shape
    m = torch.empty(K, dtype=torch.float32, device=xcal.device)
    with torch.cuda.device(xcal.device):
        _check(lib().awq_act_stats(_ptr(xcal), R, K, _ptr(m), _ptr(status), _stream(xcal)),
               "awq_act_stats")
    return m


def compute_scales(m: torch.Tensor, status: torch.Tensor | None = None) -> torch.Tensor:
    """s = sqrt(max(m, 1e-8)) / sqrt(max t * min t), float16 [K]."""
    _need(m, torch.float32, 1, "m")
    _need_status(status, m.device)
    s = torch.empty(m.shape[0], dtype=torch.float16, device=m.device)
    with torch.cuda.device(m.device):
        _check(lib().awq_compute_scales(_ptr(m), m.shape[0], _ptr(s), _ptr(status), _stream(m)),
               "awq_compute_scales")
    return s


def quantize_pack(W: torch.Tensor, s: torch.Tensor, status: torch.Tensor | None = None, out=None,
                  zero_point: bool = True):
    """Fold s into W, 4-bit group-128 quantization, packed int32.

    zero_point=True: asymmetric grid with a per-group zero point (Q, scales, zeros).
    zero_point=False: symmetric grid, zero point 8, no zeros tensor (Q, scales, None).
    """
    _need(W, torch.float16, 2, "W")
    K, N = W.shape
    dev = W.device
    _need(s, torch.float16, (K,), "s", dev)
    _need_status(status, dev)
    G = max(K // GROUP_SIZE, 1)
    if out is None:
        Q = torch.empty(K // 8, N, dtype=torch.int32, device=dev)
        sc = torch.empty(G, N, dtype=torch.float16, device=dev)
        z = (torch.empty(G, max(N // 8, 1), dtype=torch.int32, device=dev)
             if zero_point else None)
    else:
        Q, sc, z = out
        _need(Q, torch.int32, (K // 8, N), "Q", dev)
        _need(sc, torch.float16, (G, N), "scales", dev)
        if zero_point:
            _need(z, torch.int32, (G, N // 8), "zeros", dev)
    with torch.cuda.device(dev):
        if zero_point:
            _check(lib().awq_quantize_pack(_ptr(W), _ptr(s), K, N, _ptr(Q), _ptr(sc), _ptr(z),
                                           _ptr(status), _stream(W)), "awq_quantize_pack")
        else:
            _check(lib().awq_quantize_pack_symmetric(_ptr(W), _ptr(s), K, N, _ptr(Q), _ptr(sc),
                                                     _ptr(status), _stream(W)),
                   "awq_quantize_pack_symmetric")
    return Q, sc, z


def quantize_pack_clip(W: torch.Tensor, s: torch.Tensor, xcal: torch.Tensor, n_cand: int = 11,
                       status: torch.Tensor | None = None):
    """Fold s into W and quantize with weight clipping: per group and column the
    range shrink c = 1 - i/20 (i < n_cand) with the smallest output error on
    the calibration rows.  Returns (Q, scales, zeros, ratio_index int32 [K/128, N])."""
    _need(W, torch.float16, 2, "W")
    K, N = W.shape
    dev = W.device
    _need(s, torch.float16, (K,), "s", dev)
    _need(xcal, torch.float16, (None, K), "xcal", dev)
    _need_status(status, dev)
    G = max(K // GROUP_SIZE, 1)
    Q = torch.empty(K // 8, N, dtype=torch.int32, device=dev)
    sc = torch.empty(G, N, dtype=torch.float16, device=dev)
    z = torch.empty(G, max(N // 8, 1), dtype=torch.int32, device=dev)
    ri = torch.empty(G, N, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().awq_quantize_pack_clip(_ptr(W), _ptr(s), _ptr(xcal), xcal.shape[0], K, N, int(n_cand),
                                            _ptr(Q), _ptr(sc), _ptr(z), _ptr(ri), _ptr(status), _stream(W)),
               "awq_quantize_pack_clip")
    return Q, sc, z, ri


def fold_inverse_scale(a: torch.Tensor, s: torch.Tensor, status: torch.Tensor | None = None,
                       out=None) -> torch.Tensor:
    """out = fp16(a / s) per input channel; a is [K] (a norm weight) or [rows, K]."""
    if not isinstance(a, torch.Tensor) or a.dim() not in (1, 2):
        raise ValueError("a must be a [K] or [rows, K] tensor")
    a2 = a.view(1, -1) if a.dim() == 1 else a
    _need(a2, torch.float16, 2, "a")
    rows, K = a2.shape
    _need(s, torch.float16, (K,), "s", a.device)
    _need_status(status, a.device)
    if out is None:
        o = torch.empty_like(a)
    else:
        _need(out, torch.float16, tuple(a.shape), "out", a.device)
        o = out
    with torch.cuda.device(a.device):
        _check(lib().awq_fold_inverse_scale(_ptr(a2), rows, K, _ptr(s), _ptr(o), _ptr(status),
                                            _stream(a)), "awq_fold_inverse_scale")
    return o


def gemm_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().awq_w4a16_gemm_workspace_size(M, K, N))


# Zero-filled workspaces, one per (device, stream): the matmul keeps arrival
# counters in its workspace that must read zero when a call starts, and every
# call leaves them at zero again.  Calls on one stream are ordered, so they can
# share one workspace; calls on different streams get different ones.
_workspaces: dict = {}

# A call enqueues up to four kernels that pass data through its workspace, and
# ctypes lets other threads run meanwhile: the calls that use a stream's default
# workspaces take that stream's lock, so that their kernels stay together.
# (Re-entrant: an allocation inside may run a finalizer that calls the library.)
_stream_locks: dict = {}
_NO_LOCK = contextlib.nullcontext()


def _stream_lock(index: int, stream: int, workspace):
    """What a call holds while it enqueues; nothing for a workspace that the caller has brought."""
    if workspace is not None:
        return _NO_LOCK
    lock = _stream_locks.get((index, stream))
    return lock if lock is not None else _stream_locks.setdefault((index, stream), threading.RLock())


def workspace_for(device: torch.device, nbytes: int) -> torch.Tensor:
    """The zero-filled workspace this binding uses on `device`'s current stream,
    grown (as a new zero-filled buffer) when a call needs more."""
    key = (device.index, _raw_stream(device))
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def _default_workspace(dev: torch.device, M: int, need: int) -> torch.Tensor:
    """Default workspace of a product of M tokens: the stream's cached one.  A call that is being captured into
    a graph gets its own, from the graph's memory: graphs captured on one stream may be replayed at the same
    time on others, and a cached one's zeroes would be written by the first graph's replays only.  From
    64 tokens on, where the counters are used, the graph zeroes them."""
    if not _capturing():
        return workspace_for(dev, need)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    if M >= 64:
        ws[:32768].zero_()
    return ws


def scales_alpha(m: torch.Tensor, j: int, status: torch.Tensor | None = None) -> torch.Tensor:
    """Scales of grid point alpha = j/8: s = m^(j/8) normalised, float16 [K]."""
    _need(m, torch.float32, 1, "m")
    _need_status(status, m.device)
    if not 0 <= int(j) <= 8:
        raise ValueError("j must be in 0..8")
    s = torch.empty(m.shape[0], dtype=torch.float16, device=m.device)
    with torch.cuda.device(m.device):
        _check(lib().awq_scales_alpha(_ptr(m), m.shape[0], int(j), _ptr(s), _ptr(status), _stream(m)),
               "awq_scales_alpha")
    return s


def scale_search(xcal: torch.Tensor, W: torch.Tensor, status: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """Search alpha = j/8 (j = 0..8) for s = m^alpha (normalised) minimizing the
    quantized layer's output error on the calibration rows.

    Returns (s_best float16 [K], j_best int32 [1], losses float64 [9]), all on
    the device.  workspace: zero-filled uint8 of at least
    scale_search_workspace_size(R, K, N) bytes (default: a fresh one)."""
    _need(xcal, torch.float16, 2, "xcal")
    R, K = xcal.shape
    dev = xcal.device
    _need(W, torch.float16, (K, None), "W", dev)
    N = W.shape[1]
    _need_status(status, dev)
    need = scale_search_workspace_size(R, K, N)
    if need == 0:
        raise ValueError(f"unsupported shape R={R}, K={K}, N={N}")
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    else:
        _check_workspace(workspace, need, dev)
    losses = torch.empty(9, dtype=torch.float64, device=dev)
    s_best = torch.empty(K, dtype=torch.float16, device=dev)
    j_best = torch.empty(1, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().awq_scale_search(_ptr(xcal), R, K, _ptr(W), N, _ptr(losses), _ptr(s_best), _ptr(j_best),
                                      _ptr(workspace), workspace.numel(), _ptr(status), _stream(xcal)),
               "awq_scale_search")
    return s_best, j_best, losses


def scale_search_workspace_size(R: int, K: int, N: int) -> int:
    return int(lib().awq_scale_search_workspace_size(R, K, N))


def _check_weights(K, N, s, Q, scales, zeros, dev):
    if K % GROUP_SIZE or K < GROUP_SIZE:
        raise ValueError(f"K = {K} must be a positive multiple of {GROUP_SIZE}")
    if N % 8 or N < 8:
        raise ValueError(f"N = {N} must be a positive multiple of 8")
    G = K // GROUP_SIZE
    if s is not None:
        _need(s, torch.float16, (K,), "s", dev)
    _need(Q, torch.int32, (K // 8, N), "Q", dev)
    _need(scales, torch.float16, (G, N), "scales", dev)
    if zeros is not None:
        _need(zeros, torch.int32, (G, N // 8), "zeros", dev)


def _check_out(out, M, N, dev):
    _need(out, torch.float16, (M, N), "out", dev)


def _check_workspace(ws, need, dev):
    _need(ws, torch.uint8, 1, "workspace", dev)
    if ws.numel() < need:
        raise ValueError(f"workspace holds {ws.numel()} bytes, the call needs {need}")


def w4a16_gemm(X, s, Q, scales, zeros, status=None, out=None, workspace=None) -> torch.Tensor:
    """Y = (X / s) . dequant(Q), float16 [M, N].

    workspace: a uint8 CUDA tensor of at least gemm_workspace_size(M, K, N)
    bytes, zero-filled before its first use (the calls keep it that way), not
    used by two threads at once; by default a cached zero-filled workspace of
    the current stream is used, or the graph's own during capture."""
    _need(X, torch.float16, 2, "X")
    M, K = X.shape
    dev = X.device
    if not isinstance(Q, torch.Tensor) or Q.dim() != 2:
        raise ValueError("Q must be an int32 [K/8, N] tensor")
    N = Q.shape[1]
    _check_weights(K, N, s, Q, scales, zeros, dev)
    _need_status(status, dev)
    if out is None:
        Y = torch.empty(M, N, dtype=torch.float16, device=dev)
    else:
        _check_out(out, M, N, dev)
        Y = out
    with _on(dev), _stream_lock(dev.index, _raw_stream(dev), workspace):
        wsz = gemm_workspace_size(M, K, N)
        if workspace is None:
            workspace = _default_workspace(dev, M, wsz)
        else:
            _check_workspace(workspace, wsz, dev)
        _check(lib().awq_w4a16_gemm(_ptr(X), _ptr(s), _ptr(Q), _ptr(scales), _ptr(zeros), M, K, N,
                                    _ptr(Y), _ptr(workspace), workspace.numel(), _ptr(status),
                                    _stream(X)),
               "awq_w4a16_gemm")
    return Y


def w4a16_gemv(X, s, Q, scales, zeros, status=None, out=None, workspace=None) -> torch.Tensor:
    """Single-token decode: X [1, K] (or [K]) -> Y [1, N]."""
    if isinstance(X, torch.Tensor) and X.dim() == 1:
        X = X.view(1, -1)
    _need(X, torch.float16, 2, "X")
    if X.shape[0] != 1:
        raise ValueError("w4a16_gemv takes exactly one token; use w4a16_gemm")
    K = X.shape[1]
    dev = X.device
    if not isinstance(Q, torch.Tensor) or Q.dim() != 2:
        raise ValueError("Q must be an int32 [K/8, N] tensor")
    N = Q.shape[1]
    _check_weights(K, N, s, Q, scales, zeros, dev)
    _need_status(status, dev)
    if out is None:
        Y = torch.empty(1, N, dtype=torch.float16, device=dev)
    else:
        _check_out(out, 1, N, dev)
        Y = out
    with _on(dev), _stream_lock(dev.index, _raw_stream(dev), workspace):
        wsz = int(lib().awq_w4a16_gemv_workspace_size(K, N))
        if workspace is None:
            workspace = _default_workspace(dev, 1, wsz)
        else:
            _check_workspace(workspace, wsz, dev)
        _check(lib().awq_w4a16_gemv(_ptr(X), _ptr(s), _ptr(Q), _ptr(scales), _ptr(zeros), K, N,
                                    _ptr(Y), _ptr(workspace), workspace.numel(), _ptr(status),
                                    _stream(X)), "awq_w4a16_gemv")
    return Y


def _check_epilogue(N, bias, act, gated, dev):
    """Checks the layer side of an epilogue; returns (act code, gated flag, columns of Y)."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(k for k in ACTIVATIONS if k)} or None, got {act!r}")
    if bias is not None:
        _need(bias, torch.float16, (N,), "bias", dev)
    if gated and N % 16:
        raise ValueError(f"a gated product needs N = {N} to be a multiple of 16")
    return ACTIVATIONS[act], int(bool(gated)), N // 2 if gated else N


def w4a16_gemm_epilogue(X, s, Q, scales, zeros, bias=None, act=None, gated=False, residual=None, status=None,
                        out=None, workspace=None) -> torch.Tensor:
    """Y = act((X / s) . dequant(Q) + bias) + residual, rounded once to float16.

    act: None, "relu", "silu", "gelu" or "gelu_tanh".
    gated: columns 2j are the gate of columns 2j + 1 (see interleave_gate_up): Y is
    act(t[:, 0::2]) * t[:, 1::2] + residual, [M, N/2].
    residual: float16 of Y's shape; out may be residual itself.
    workspace: as for w4a16_gemm; by default the stream's cached one, or the graph's own during capture."""
    _need(X, torch.float16, 2, "X")
    M, K = X.shape
    dev = X.device
    if not isinstance(Q, torch.Tensor) or Q.dim() != 2:
        raise ValueError("Q must be an int32 [K/8, N] tensor")
    N = Q.shape[1]
    _check_weights(K, N, s, Q, scales, zeros, dev)
    code, gate, cols = _check_epilogue(N, bias, act, gated, dev)
    if residual is not None:
        _need(residual, torch.float16, (M, cols), "residual", dev)
    _need_status(status, dev)
    if out is None:
        Y = torch.empty(M, cols, dtype=torch.float16, device=dev)
    else:
        _check_out(out, M, cols, dev)
        Y = out
    with _on(dev), _stream_lock(dev.index, _raw_stream(dev), workspace):
        wsz = gemm_workspace_size(M, K, N)
        if workspace is None:
            workspace = _default_workspace(dev, M, wsz)
        else:
            _check_workspace(workspace, wsz, dev)
        _check(lib().awq_w4a16_gemm_epilogue(_ptr(X), _ptr(s), _ptr(Q), _ptr(scales), _ptr(zeros), M, K, N,
                                             _ptr(bias), code, gate, _ptr(residual), _ptr(Y), _ptr(workspace),
                                             workspace.numel(), _ptr(status), _stream(X)),
               "awq_w4a16_gemm_epilogue")
    return Y


def interleave_gate_up(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """The weight [K, 2 I] of a gated product from its gate and up weights [K, I]: column 2j from the gate,
    column 2j + 1 from up.  Quantize the result and pass gated=True.  Biases [I] interleave the same way."""
    if gate.shape != up.shape:
        raise ValueError(f"gate {tuple(gate.shape)} and up {tuple(up.shape)} must have one shape")
    return torch.stack((gate, up), dim=-1).flatten(-2)


class QuantLinear:
    """A quantized linear layer ("Awq Quantization", "WQLinear Kernel
    Variants": one module whose forward runs the fused-dequantization kernel).

    The weights (Q, scales, zeros, s) are checked once here; a call checks
    only X and the output, and passes prepared pointers to the C ABI.

    bias, act and gated fuse what follows the product (w4a16_gemm_epilogue);
    a call may add a residual: layer(X, residual=r)."""

    def __init__(self, Q, scales, zeros=None, s=None, bias=None, act=None, gated=False):
        if not isinstance(Q, torch.Tensor) or Q.dim() != 2:
            raise ValueError("Q must be an int32 [K/8, N] tensor")
        self.K, self.N = Q.shape[0] * 8, Q.shape[1]
        self.device = Q.device
        _check_weights(self.K, self.N, s, Q, scales, zeros, self.device)
        self.Q, self.scales, self.zeros, self.s = Q, scales, zeros, s
        self._wptrs = (_ptr(s), _ptr(Q), _ptr(scales), _ptr(zeros))
        self.bias, self.act, self.gated = bias, act, bool(gated)
        self._act, self._gate, self.out_features = _check_epilogue(self.N, bias, act, gated, self.device)
        self._plain = bias is None and self._act == 0 and not gated
        self._bptr = _ptr(bias)
        self._dev_index = self.device.index if self.device.index is not None else torch.cuda.current_device()
        self._lib = lib()

    def __call__(self, X, out=None, status=None, workspace=None, residual=None) -> torch.Tensor:
        if not isinstance(X, torch.Tensor) or X.dtype != torch.float16 or X.dim() != 2 \
                or X.shape[1] != self.K or X.device != self.device or not X.is_contiguous():
            raise ValueError(f"X must be a contiguous float16 [M, {self.K}] tensor on {self.device}")
        M = X.shape[0]
        cols = self.out_features
        if out is None:
            out = torch.empty(M, cols, dtype=torch.float16, device=self.device)
        elif out.dtype != torch.float16 or tuple(out.shape) != (M, cols) or out.device != self.device \
                or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous float16 [{M}, {cols}] tensor on {self.device}")
        if residual is not None and (
                residual.dtype != torch.float16 or tuple(residual.shape) != (M, cols)
                or residual.device != self.device or not residual.is_contiguous()):
            raise ValueError(f"residual must be a contiguous float16 [{M}, {cols}] tensor on {self.device}")
        if status is not None:
            _need_status(status, self.device)
        stream = torch._C._cuda_getCurrentRawStream(self._dev_index)
        wsz = self._lib.awq_w4a16_gemm_workspace_size(M, self.K, self.N)
        plain = self._plain and residual is None
        s, q, sc, z = self._wptrs
        with _stream_lock(self._dev_index, stream, workspace):
            if workspace is not None:
                _check_workspace(workspace, wsz, self.device)
            else:
                workspace = _default_workspace(self.device, M, wsz)
            if not plain:
                _call(self.device, "awq_w4a16_gemm_epilogue", self._lib.awq_w4a16_gemm_epilogue, X.data_ptr(), s, q, sc,
                      z, M, self.K, self.N, self._bptr, self._act, self._gate, _ptr(residual), out.data_ptr(),
                      workspace.data_ptr(), workspace.numel(), _ptr(status), stream)
            else:
                _call(self.device, "awq_w4a16_gemm", self._lib.awq_w4a16_gemm, X.data_ptr(), s, q, sc, z, M, self.K,
                      self.N, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _ptr(status), stream)
        return out


# ---------------------------------------------------------------- paged 4-bit key/value cache
KV4_PAGE_SIZES = (16, 32, 64, 128, 256)


def kv4_page_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of one page for one head."""
    n = int(lib().awq_kv4_page_bytes(page_size, head_dim))
    if n == 0:
        raise ValueError(f"page_size must be one of {KV4_PAGE_SIZES} and head_dim 64 or 128, "
                         f"got {page_size} and {head_dim}")
    return n


def _match(t, dtype, shape, name, dev):
    """_need for the calls of a step: one test when all is well."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _need(t, dtype, shape, name, dev)


class KV4Pages:
    """Pages of a 4-bit key/value cache and the requests that hold them; shared by the caches of all layers.

    num_pages pages of page_size tokens (16, 32, 64, 128 or 256); max_requests rows of at most max_pages
    pages.  State on the device, all int32: block_table [max_requests, max_pages], lens [max_requests],
    free_pages [num_pages] with free_count [1] (a stack).  Given tensors are used as they are; by default every page is
    free.  The state tensors may be written at any time but not replaced: calls and captured graphs keep their
    addresses."""

    def __init__(self, num_pages, page_size, max_requests, max_pages, device="cuda", block_table=None, lens=None,
                 free_pages=None, free_count=None):
        if page_size not in KV4_PAGE_SIZES:
            raise ValueError(f"page_size must be one of {KV4_PAGE_SIZES}, got {page_size}")
        if not 1 <= max_requests <= KV4_MAX_REQUESTS:
            raise ValueError(f"max_requests must be in 1..{KV4_MAX_REQUESTS}, got {max_requests}")
        if num_pages < 1 or num_pages >= 2**31 or max_pages < 1 or max_pages * page_size >= 2**31:
            raise ValueError(f"num_pages = {num_pages} and max_pages * page_size = {max_pages * page_size} must be "
                             "positive and below 2**31")
        if (free_pages is None) != (free_count is None):
            raise ValueError("free_pages and free_count go together")
        first = next((t for t in (block_table, lens, free_pages) if isinstance(t, torch.Tensor)), None)
        dev = first.device if first is not None else torch.device(device)
        if dev.type != "cuda":
            raise TypeError(f"the pages live on a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.num_pages, self.page_size = dev, num_pages, page_size
        self.max_requests, self.max_pages = max_requests, max_pages
        i32 = dict(dtype=torch.int32, device=dev)
        self.block_table = block_table if block_table is not None else \
            torch.full((max_requests, max_pages), -1, **i32)
        self.lens = lens if lens is not None else torch.zeros(max_requests, **i32)
        self.free_pages = free_pages if free_pages is not None else torch.arange(num_pages - 1, -1, -1, **i32)
        self.free_count = free_count if free_count is not None else torch.full((1,), num_pages, **i32)
        _need(self.block_table, torch.int32, (max_requests, max_pages), "block_table", dev)
        _need(self.lens, torch.int32, (max_requests,), "lens", dev)
        _need(self.free_pages, torch.int32, (num_pages,), "free_pages", dev)
        _need(self.free_count, torch.int32, (1,), "free_count", dev)
        self._lib = lib()
        self._state = (self.block_table.data_ptr(), max_pages, self.free_pages.data_ptr(), self.free_count.data_ptr(),
                       num_pages)

    def reserve(self, new_lens, total, next_lens=None, next_free=None, out=None, status=None):
        """Pages and slots for new_lens[b] new tokens of each request b (int32 [max_requests]).

        total: rows of the step, at least the sum of new_lens (the rows behind are padding).
        Returns (slots int64 [total], positions int32 [total], cu int32 [max_requests + 1]); slots and positions are
        -1 in the padding.  The new lengths and free count go to next_lens and next_free (default: in place).
        status receives ERR_CAPACITY when the free pages do not suffice, ERR_RANGE for impossible lengths; then nothing
        is reserved and every slot is -1.  ERR_RANGE also for a page outside the cache, held or free: its tokens get
        slot -1, the others their slots."""
        dev, B = self.device, self.max_requests
        _match(new_lens, torch.int32, (B,), "new_lens", dev)
        if not 1 <= total < 2**31:
            raise ValueError(f"total must be in 1..2**31 - 1, got {total}")
        if next_lens is None:
            next_lens = self.lens
        else:
            _match(next_lens, torch.int32, (B,), "next_lens", dev)
        if next_free is None:
            next_free = self.free_count
        else:
            _match(next_free, torch.int32, (1,), "next_free", dev)
        if out is None:
            slots = torch.empty(total, dtype=torch.int64, device=dev)
            positions, cu = self.lens.new_empty(total), self.lens.new_empty(B + 1)
        else:
            slots, positions, cu = out
            _match(slots, torch.int64, (total,), "slots", dev)
            _match(positions, torch.int32, (total,), "positions", dev)
            _match(cu, torch.int32, (B + 1,), "cu", dev)
        if status is not None:
            _need_status(status, dev)
        _call(dev, "awq_kv4_reserve", self._lib.awq_kv4_reserve, new_lens.data_ptr(), self.lens.data_ptr(), B,
              self.page_size, *self._state, total, slots.data_ptr(), positions.data_ptr(), cu.data_ptr(),
              next_lens.data_ptr(), next_free.data_ptr(), _ptr(status), _raw_stream(dev))
        return slots, positions, cu

    def release(self, done, status=None):
        """Ends the requests with done[b] != 0 (int32 [max_requests]): their pages return to the stack.

        Every page that such a request holds must be in its row of the table and in no other request's.  Entries of -1
        are passed over: pages before a sliding window may be given back earlier, by writing them to
        free_pages[free_count], raising free_count and setting their entries to -1."""
        dev = self.device
        _match(done, torch.int32, (self.max_requests,), "done", dev)
        if status is not None:
            _need_status(status, dev)
        _call(dev, "awq_kv4_release", self._lib.awq_kv4_release, done.data_ptr(), self.lens.data_ptr(),
              self.max_requests, self.page_size, *self._state, _ptr(status), _raw_stream(dev))


class KV4Cache:
    """Keys and values of one layer in 4 bits, on the pages of a KV4Pages.

    data: uint8 [num_pages, kv_heads, kv4_page_bytes(page_size, head_dim)] (default: a zeroed one);
    like the state of the pages it is updated in place, never replaced."""

    def __init__(self, pages: KV4Pages, kv_heads: int, head_dim: int, data=None):
        if not 1 <= kv_heads <= 1024:
            raise ValueError(f"kv_heads must be in 1..1024, got {kv_heads}")
        self.pages, self.kv_heads, self.head_dim = pages, kv_heads, head_dim
        size = kv4_page_bytes(pages.page_size, head_dim)
        shape = (pages.num_pages, kv_heads, size)
        self.data = data if data is not None else torch.zeros(shape, dtype=torch.uint8, device=pages.device)
        _need(self.data, torch.uint8, shape, "data", pages.device)
        self._lib = lib()
        self._workspace_size = int(self._lib.awq_kv4_attention_workspace_size(head_dim))
        # the cache as the store's and load's calls and as the attention's call name it
        self._place = (kv_heads, head_dim, self.data.data_ptr(), pages.num_pages, pages.page_size)
        self._read = (self.data.data_ptr(), pages.num_pages, pages.page_size, kv_heads, head_dim,
                      pages.block_table.data_ptr(), pages.max_pages, pages.lens.data_ptr())

    def _rows(self, x, name):
        """(T, row stride) of keys or values [T, kv_heads, head_dim] or [T, kv_heads * head_dim], rows apart by any
        multiple of 8 elements."""
        H, D = self.kv_heads, self.head_dim
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if x.dtype is not torch.float16:
            raise TypeError(f"{name} must be {torch.float16}, got {x.dtype}")
        if x.device != self.pages.device:
            raise ValueError(f"{name} is on {x.device}, expected {self.pages.device}")
        sh, st = x.shape, x.stride()
        if len(sh) == 3 and sh[1] == H and sh[2] == D:
            if st[2] != 1 or (st[1] != D and H > 1):
                raise ValueError(f"the heads of {name} must be contiguous, got strides {st}")
        elif not (len(sh) == 2 and sh[1] == H * D and st[1] == 1):
            raise ValueError(f"{name} must have shape (T, {H}, {D}) or (T, {H * D}) with contiguous rows, got {tuple(sh)}")
        T = sh[0]
        if T == 1:
            return T, H * D
        if st[0] < H * D or st[0] % 8:
            raise ValueError(f"rows of {name} must be at least {H * D} elements apart, by a multiple of 8, got {st[0]}")
        return T, st[0]

    def append(self, k, v, slots, status=None):
        """Quantizes keys and values [T, kv_heads, head_dim] (float16; rows may be slices of a fused projection's) into
        slots (int64 [T]; negative: not stored)."""
        T, ks = self._rows(k, "k")
        Tv, vs = self._rows(v, "v")
        dev = self.pages.device
        if T != Tv:
            raise ValueError(f"k has {T} rows, v {Tv}")
        _match(slots, torch.int64, (T,), "slots", dev)
        if status is not None:
            _need_status(status, dev)
        if T == 0:
            return
        _call(dev, "awq_kv4_append", self._lib.awq_kv4_append, k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), T,
              *self._place, _ptr(status), _raw_stream(dev))

    def load(self, slots, out=None, status=None):
        """The stored keys and values of slots (int64 [T]): (k, v) float16 [T, kv_heads, head_dim]; zeros for a negative
        slot."""
        dev = self.pages.device
        T = slots.numel() if isinstance(slots, torch.Tensor) else 0
        _match(slots, torch.int64, (T,), "slots", dev)
        shape = (T, self.kv_heads, self.head_dim)
        if out is None:
            k = torch.empty(shape, dtype=torch.float16, device=dev)
            v = torch.empty(shape, dtype=torch.float16, device=dev)
        else:
            k, v = out
            _match(k, torch.float16, shape, "k", dev)
            _match(v, torch.float16, shape, "v", dev)
        if status is not None:
            _need_status(status, dev)
        if T == 0:
            return k, v
        _call(dev, "awq_kv4_load", self._lib.awq_kv4_load, slots.data_ptr(), T, *self._place, k.data_ptr(), v.data_ptr(),
              _ptr(status), _raw_stream(dev))
        return k, v

    def attention(self, q, cu=None, max_new=1, scale=None, window=0, out=None, status=None, workspace=None):
        """Causal attention of q [T, q_heads, head_dim] (float16; rows may be slices of a fused projection's) over the
        cached tokens of the pages' requests, the new tokens among them (append first).

        cu: int32 [max_requests + 1], the query rows of each request (from reserve); None: one query per request.
        max_new: the most queries of one request.  scale: default head_dim ** -0.5.
        window: positions seen, 0 for all; pages wholly before it may be gone from the table (-1).
        Returns [T, q_heads, head_dim]; rows of no request are not written.
        AwqError (ERR_SHAPE) for bounds whose work is not counted in 32 bits: max_requests * kv_heads *
        (1 to 3, by rows of a request) * (max_pages * page_size / 64 + 8) has to stay below 2**32.
        workspace: uint8 of kv4_attention_workspace_size(head_dim) bytes, not used by two threads at once; by default
        the stream's cached one, or the graph's own during capture."""
        p = self.pages
        dev, D = p.device, self.head_dim
        if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[2] != D or q.dtype is not torch.float16 \
                or q.device != dev:
            raise ValueError(f"q must be a float16 [T, q_heads, {D}] tensor on {dev}")
        T, H, _ = q.shape
        st = q.stride()
        if st[2] != 1 or (st[1] != D and H > 1) or (T > 1 and (st[0] < H * D or st[0] % 8)):
            raise ValueError(f"the heads of q must be contiguous and its rows a multiple of 8 elements apart, got strides {st}")
        if H == 0 or H % self.kv_heads:
            raise ValueError(f"q has {H} heads, not a multiple of the cache's {self.kv_heads}")
        if cu is not None:
            _match(cu, torch.int32, (p.max_requests + 1,), "cu", dev)
        elif T < p.max_requests:
            raise ValueError(f"without cu, q needs a row for each of the {p.max_requests} requests, got {T}")
        if max_new < 1 or window < 0:
            raise ValueError(f"max_new must be at least 1 and window at least 0, got {max_new} and {window}")
        if out is None:
            out = torch.empty((T, H, D), dtype=torch.float16, device=dev)
        else:
            _match(out, torch.float16, (T, H, D), "out", dev)
        if status is not None:
            _need_status(status, dev)
        if T == 0:
            return out
        stream = _raw_stream(dev)
        with _stream_lock(dev.index, stream, workspace):
            if workspace is not None:
                _check_workspace(workspace, self._workspace_size, dev)
            elif _capturing():
                workspace = torch.empty(self._workspace_size, dtype=torch.uint8, device=dev)
            else:
                workspace = _kv4_workspace(dev, stream, self._workspace_size)
            _call(dev, "awq_kv4_attention", self._lib.awq_kv4_attention, q.data_ptr(), st[0] if T > 1 else H * D, T, H,
                  *self._read, _ptr(cu), p.max_requests, max_new, D ** -0.5 if scale is None else scale, window,
                  out.data_ptr(), workspace.data_ptr(), workspace.numel(), _ptr(status), stream)
        return out


def kv4_attention_workspace_size(head_dim: int) -> int:
    return int(lib().awq_kv4_attention_workspace_size(head_dim))


# The attention's workspaces, one per (device, stream), apart from the matmul's:
# they are overwritten and never need zeroes.
_kv4_workspaces: dict = {}


def _kv4_workspace(device: torch.device, stream: int, nbytes: int) -> torch.Tensor:
    key = (device.index, stream)
    ws = _kv4_workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _kv4_workspaces[key] = ws
    return ws
