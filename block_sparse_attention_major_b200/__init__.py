"""Python binding of libbsa, the B200 block-sparse video attention library.

Argument marshalling only: every step of the path runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream. There is no CPU fallback: if
libbsa.so is missing or the device is not a B200, the calls raise.

Entry points (same names as the C ABI in include/bsa.h):
    reorder(g, x)                   raster [B,N,H,d] -> tile-major [B,H,NT,64,d]
    reorder_pool(g, x)              the same, plus the per-tile means fp32 [B,H,NT,d]
    unreorder(g, xt)                the inverse
    build_mask(g, p, qt, kt, difficulty)     -> (mask uint32 [B,H,NQT,W], kv_count int32)
    build_mask_pooled(g, p, qbar, kbar, difficulty)   the same from the per-tile means
    sparse_attn_fwd(g, qt, kt, vt, mask, kv_count)  -> (out bf16 [B,N,H,d], lse fp32 [B,H,N])
    sparse_attn_fwd_token(g, qt, kt, vt, mask, kv_count, dense, token_radius)
                                    the same under a token-level circular support
    forward(g, p, q, k, v, difficulty)       the whole path, raster in, raster out
    cross_attn_fwd(g, q, k, v, kv_len, key_mask)    attention to an encoder's states of another
                                    length -> (out bf16 [B,N,H,d], lse fp32 [B,H,N])
    cross_attn_bwd(g, q, k, v, out, lse, dout, ...)    its gradients -> (dq, dk, dv)
    cross_forward(g, q, k, v, ..., qk_norm)  the norm of Q and K per head, then that attention
    layer_norm_fwd(x, weight, bias)          -> (y, mean, rstd), over the last axis
    layer_norm_bwd(x, dy, mean, rstd, weight)    -> (dx, dweight, dbias)

No call takes part in autograd: outputs have no grad_fn, whatever the inputs require. Gradients
are those that the _bwd calls return.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsa.so")

BSA_OK = 0
STATUS_NAMES = {0: "BSA_OK", 1: "BSA_ERR_INVALID_ARG", 2: "BSA_ERR_WORKSPACE",
                3: "BSA_ERR_UNSUPPORTED_DEVICE", 4: "BSA_ERR_CUDA"}
KERR_WAIT_TIMEOUT, KERR_BAD_UNIT, KERR_BAD_MASK = 1, 2, 4


class bsa_geom(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("T", ctypes.c_int), ("Hs", ctypes.c_int), ("Ws", ctypes.c_int)]


class bsa_mask_params(ctypes.Structure):
    _fields_ = [("window_kind", ctypes.c_int), ("radius", ctypes.c_int), ("topk", ctypes.c_int),
                ("dense_fraction", ctypes.c_float), ("budget_mode", ctypes.c_int),
                ("budget_target", ctypes.c_float)]


class bsa_cross_geom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "Hkv", "d", "N", "M")]


class bsa_cross_strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_longlong * 3) for n in ("q", "k", "v")]


class bsa_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("C", ctypes.c_int), ("items", ctypes.c_int),
                ("w_per_item", ctypes.c_int), ("x_type", ctypes.c_int), ("y_type", ctypes.c_int),
                ("w_type", ctypes.c_int), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class BsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")
        self.status = status


_lib = None
_lib_lock = threading.Lock()


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libbsa.so (built in-tree by _build.py); raises if it is missing."""
    global _lib
    with _lib_lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libbsa.so not found at {p}: run `python -m "
                               "block_sparse_attention_major_b200._build` first")
        lib = ctypes.CDLL(p)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        G, P = ctypes.POINTER(bsa_geom), ctypes.POINTER(bsa_mask_params)
        lib.bsa_status_string.restype = ctypes.c_char_p
        lib.bsa_status_string.argtypes = [ctypes.c_int]
        lib.bsa_tile_grid.restype = ctypes.c_int
        lib.bsa_tile_grid.argtypes = [G] + [ctypes.POINTER(ctypes.c_int)] * 4
        lib.bsa_workspace_bytes.restype = sz
        lib.bsa_workspace_bytes.argtypes = [G, P]
        lib.bsa_clear_error.restype = ctypes.c_int
        lib.bsa_clear_error.argtypes = [vp, vp]
        lib.bsa_reorder.restype = ctypes.c_int
        lib.bsa_reorder.argtypes = [G, vp, vp, vp]
        lib.bsa_unreorder.restype = ctypes.c_int
        lib.bsa_unreorder.argtypes = [G, vp, vp, vp]
        lib.bsa_reorder_pool.restype = ctypes.c_int
        lib.bsa_reorder_pool.argtypes = [G, vp, vp, vp, vp]
        lib.bsa_build_mask_pooled.restype = ctypes.c_int
        lib.bsa_build_mask_pooled.argtypes = [G, P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.bsa_build_mask.restype = ctypes.c_int
        lib.bsa_build_mask.argtypes = [G, P, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.bsa_sparse_attn_fwd.restype = ctypes.c_int
        lib.bsa_sparse_attn_fwd.argtypes = [G, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, sz, vp]
        lib.bsa_sparse_attn_fwd_token.restype = ctypes.c_int
        lib.bsa_sparse_attn_fwd_token.argtypes = [G, vp, vp, vp, vp, vp, vp, ctypes.c_int, ctypes.c_float, vp,
                                                  vp, vp, sz, vp]
        lib.bsa_route_flags_offset.restype = sz
        lib.bsa_route_flags_offset.argtypes = [G]
        lib.bsa_sparse_attn_fwd_fixed_scratch.restype = ctypes.c_int
        lib.bsa_sparse_attn_fwd_fixed_scratch.argtypes = [G, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                                          vp, vp]
        X, T = ctypes.POINTER(bsa_cross_geom), ctypes.POINTER(bsa_cross_strides)
        lib.bsa_cross_workspace_bytes.restype = sz
        lib.bsa_cross_workspace_bytes.argtypes = [X]
        lib.bsa_cross_attn_fwd.restype = ctypes.c_int
        lib.bsa_cross_attn_fwd.argtypes = [X, T] + [vp] * 5 + [ctypes.c_float] + [vp] * 3 + [sz, vp]
        lib.bsa_cross_attn_bwd.restype = ctypes.c_int
        lib.bsa_cross_attn_bwd.argtypes = [X, T] + [vp] * 8 + [ctypes.c_float] + [vp] * 4 + [sz, vp]
        N = ctypes.POINTER(bsa_norm_shape)
        lib.bsa_layer_norm_fwd.restype = ctypes.c_int
        lib.bsa_layer_norm_fwd.argtypes = [N] + [vp] * 7
        lib.bsa_layer_norm_workspace_bytes.restype = sz
        lib.bsa_layer_norm_workspace_bytes.argtypes = [N]
        lib.bsa_layer_norm_bwd.restype = ctypes.c_int
        lib.bsa_layer_norm_bwd.argtypes = [N] + [vp] * 9 + [sz, vp]
        lib.bsa_launch_count.restype = ctypes.c_uint64
        lib.bsa_launch_count.argtypes = []
        lib.bsa_selftest_bounded_wait.restype = ctypes.c_int
        lib.bsa_selftest_bounded_wait.argtypes = [ctypes.c_longlong, vp, vp]
        lib.bsa_selftest_cross_wait.restype = ctypes.c_int
        lib.bsa_selftest_cross_wait.argtypes = [vp, vp]
        if path is None:
            _lib = lib
        return lib


@dataclass(frozen=True)
class Geometry:
    B: int
    H: int
    d: int
    T: int
    Hs: int
    Ws: int

    @property
    def N(self) -> int:
        return self.T * self.Hs * self.Ws

    @property
    def tiles(self) -> tuple[int, int, int]:
        return (-(-self.T // 4), -(-self.Hs // 4), -(-self.Ws // 4))

    @property
    def NT(self) -> int:
        a, b, c = self.tiles
        return a * b * c

    @property
    def NW(self) -> int:
        return -(-self.NT // 32)

    def c(self) -> bsa_geom:
        return bsa_geom(self.B, self.H, self.d, self.T, self.Hs, self.Ws)


@dataclass(frozen=True)
class CrossGeometry:
    """Shape of an attention call to an encoder's states: B items of N query tokens with H heads,
    and M encoder states with Hkv key heads (a divisor of H)."""

    B: int
    H: int
    Hkv: int
    d: int
    N: int
    M: int

    def c(self) -> bsa_cross_geom:
        return bsa_cross_geom(self.B, self.H, self.Hkv, self.d, self.N, self.M)


@dataclass(frozen=True)
class MaskParams:
    window_kind: int = 0
    radius: int = 1
    topk: int = 0
    dense_fraction: float = 0.0
    budget_mode: int = 0
    budget_target: float = 0.0

    def c(self) -> bsa_mask_params:
        return bsa_mask_params(self.window_kind, self.radius, self.topk, self.dense_fraction,
                               self.budget_mode, self.budget_target)


def _stream(stream, device: torch.device) -> ctypes.c_void_p:
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def _device_of(*tensors: torch.Tensor | None) -> torch.device:
    """The one device of the given tensors (None entries skipped). The library launches on
    the current device with the pointers it is given, so tensors of two devices, or of a
    device other than the one the call runs on, are refused here."""
    devs = [t.device for t in tensors if t is not None]
    if not devs or any(d != devs[0] for d in devs):
        raise ValueError(f"tensors of one call must share one device, got {sorted(set(map(str, devs)))}")
    return devs[0]


def _run(what: str, device: torch.device, stream, call) -> None:
    """call(stream_handle) with `device` current, so that the library's launches, its
    device queries and the stream all refer to the device that holds the tensors."""
    with torch.cuda.device(device):
        _check(call(_stream(stream, device)), what)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, dtype, shape, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_ws(ws: torch.Tensor) -> None:
    if (not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.dtype != torch.uint8 or ws.dim() != 1
            or not ws.is_contiguous()):
        raise ValueError("ws must be a contiguous 1-D uint8 CUDA tensor (see alloc_workspace)")


def _check(status: int, what: str) -> None:
    if status != BSA_OK:
        raise BsaError(status, what)


def workspace_bytes(g: Geometry, p: MaskParams | None = None) -> int:
    pc = p.c() if p is not None else None
    return int(load_library().bsa_workspace_bytes(ctypes.byref(g.c()),
                                                  ctypes.byref(pc) if pc is not None else None))


def alloc_workspace(g: Geometry, device=None) -> torch.Tensor:
    """A zeroed device workspace (byte 0 = kernel error word)."""
    n = workspace_bytes(g)
    if n == 0:
        raise ValueError("invalid geometry")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def read_error(ws: torch.Tensor) -> int:
    """The kernel error word (synchronises the current stream)."""
    return int(ws[:4].view(torch.int32).item()) & 0xFFFFFFFF


def clear_error(ws: torch.Tensor, stream=None) -> None:
    _need_ws(ws)
    _run("bsa_clear_error", ws.device, stream, lambda s: load_library().bsa_clear_error(_ptr(ws), s))


def launch_count() -> int:
    return int(load_library().bsa_launch_count())


def selftest_bounded_wait(err: torch.Tensor, limit_cycles: int = 20_000_000, stream=None) -> None:
    """Run the bounded-wait self-test: a wait that nothing completes gives up after
    limit_cycles SM cycles and sets BSA_KERR_WAIT_TIMEOUT in err (int32 [1], device)."""
    _need(err, torch.int32, (1,), "err")
    _run("bsa_selftest_bounded_wait", err.device, stream,
         lambda s: load_library().bsa_selftest_bounded_wait(ctypes.c_longlong(limit_cycles), _ptr(err), s))


def selftest_cross_wait(err: torch.Tensor, stream=None) -> None:
    """Run the self-test of the cross attention's bounded wait: half the warps of a group wait for an
    arrival that never comes, give up and take the others with them; KERR_WAIT_TIMEOUT in err
    (int32 [1], device), KERR_BAD_UNIT where a thread was told to carry on."""
    _need(err, torch.int32, (1,), "err")
    _run("bsa_selftest_cross_wait", err.device, stream, lambda s: load_library().bsa_selftest_cross_wait(_ptr(err), s))


def reorder(g: Geometry, x: torch.Tensor, xt: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need(x, torch.bfloat16, (g.B, g.N, g.H, g.d), "x")
    if xt is None:
        xt = torch.empty((g.B, g.H, g.NT, 64, g.d), dtype=torch.bfloat16, device=x.device)
    _need(xt, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), "xt")
    _run("bsa_reorder", _device_of(x, xt), stream,
         lambda s: load_library().bsa_reorder(ctypes.byref(g.c()), _ptr(x), _ptr(xt), s))
    return xt


def reorder_pool(g: Geometry, x: torch.Tensor, xt: torch.Tensor | None = None,
                 xbar: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Tile-major reorder and the per-tile means of the valid tokens, in one pass."""
    _need(x, torch.bfloat16, (g.B, g.N, g.H, g.d), "x")
    if xt is None:
        xt = torch.empty((g.B, g.H, g.NT, 64, g.d), dtype=torch.bfloat16, device=x.device)
    if xbar is None:
        xbar = torch.empty((g.B, g.H, g.NT, g.d), dtype=torch.float32, device=x.device)
    _need(xt, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), "xt")
    _need(xbar, torch.float32, (g.B, g.H, g.NT, g.d), "xbar")
    _run("bsa_reorder_pool", _device_of(x, xt, xbar), stream,
         lambda s: load_library().bsa_reorder_pool(ctypes.byref(g.c()), _ptr(x), _ptr(xt), _ptr(xbar), s))
    return xt, xbar


def unreorder(g: Geometry, xt: torch.Tensor, x: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need(xt, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), "xt")
    if x is None:
        x = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=xt.device)
    _need(x, torch.bfloat16, (g.B, g.N, g.H, g.d), "x")
    _run("bsa_unreorder", _device_of(xt, x), stream,
         lambda s: load_library().bsa_unreorder(ctypes.byref(g.c()), _ptr(xt), _ptr(x), s))
    return x


def build_mask(g: Geometry, p: MaskParams, qt: torch.Tensor, kt: torch.Tensor,
               difficulty: torch.Tensor, mask: torch.Tensor | None = None,
               kv_count: torch.Tensor | None = None, ws: torch.Tensor | None = None,
               stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    _need(qt, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), "qt")
    _need(kt, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), "kt")
    _need(difficulty, torch.float32, (g.B, g.NT), "difficulty")
    dev = qt.device
    if mask is None:
        mask = torch.empty((g.B, g.H, g.NT, g.NW), dtype=torch.int32, device=dev)
    if kv_count is None:
        kv_count = torch.empty((g.B, g.H, g.NT), dtype=torch.int32, device=dev)
    _need(mask, torch.int32, (g.B, g.H, g.NT, g.NW), "mask")
    _need(kv_count, torch.int32, (g.B, g.H, g.NT), "kv_count")
    if ws is None:
        ws = alloc_workspace(g, dev)
    _need_ws(ws)
    pc = p.c()
    _run("bsa_build_mask", _device_of(qt, kt, difficulty, mask, kv_count, ws), stream,
         lambda s: load_library().bsa_build_mask(ctypes.byref(g.c()), ctypes.byref(pc), _ptr(qt), _ptr(kt),
                                                 _ptr(difficulty), _ptr(mask), _ptr(kv_count), _ptr(ws),
                                                 ctypes.c_size_t(ws.numel()), s))
    return mask, kv_count


def build_mask_pooled(g: Geometry, p: MaskParams, qbar: torch.Tensor, kbar: torch.Tensor,
                      difficulty: torch.Tensor, mask: torch.Tensor | None = None,
                      kv_count: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """build_mask from the per-tile means that reorder_pool wrote."""
    _need(qbar, torch.float32, (g.B, g.H, g.NT, g.d), "qbar")
    _need(kbar, torch.float32, (g.B, g.H, g.NT, g.d), "kbar")
    _need(difficulty, torch.float32, (g.B, g.NT), "difficulty")
    dev = qbar.device
    if mask is None:
        mask = torch.empty((g.B, g.H, g.NT, g.NW), dtype=torch.int32, device=dev)
    if kv_count is None:
        kv_count = torch.empty((g.B, g.H, g.NT), dtype=torch.int32, device=dev)
    _need(mask, torch.int32, (g.B, g.H, g.NT, g.NW), "mask")
    _need(kv_count, torch.int32, (g.B, g.H, g.NT), "kv_count")
    if ws is None:
        ws = alloc_workspace(g, dev)
    _need_ws(ws)
    pc = p.c()
    _run("bsa_build_mask_pooled", _device_of(qbar, kbar, difficulty, mask, kv_count, ws), stream,
         lambda s: load_library().bsa_build_mask_pooled(ctypes.byref(g.c()), ctypes.byref(pc), _ptr(qbar),
                                                        _ptr(kbar), _ptr(difficulty), _ptr(mask),
                                                        _ptr(kv_count), _ptr(ws), ctypes.c_size_t(ws.numel()),
                                                        s))
    return mask, kv_count


def sparse_attn_fwd(g: Geometry, qt: torch.Tensor, kt: torch.Tensor, vt: torch.Tensor,
                    mask: torch.Tensor, kv_count: torch.Tensor, scale: float | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None, want_lse: bool = True,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt)):
        _need(t, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), name)
    _need(mask, torch.int32, (g.B, g.H, g.NT, g.NW), "mask")
    _need(kv_count, torch.int32, (g.B, g.H, g.NT), "kv_count")
    dev = qt.device
    if out is None:
        out = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, (g.B, g.N, g.H, g.d), "out")
    if want_lse and lse is None:
        lse = torch.empty((g.B, g.H, g.N), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, torch.float32, (g.B, g.H, g.N), "lse")
    if ws is None:
        ws = alloc_workspace(g, dev)
    _need_ws(ws)
    sc = 1.0 / math.sqrt(g.d) if scale is None else float(scale)
    _run("bsa_sparse_attn_fwd", _device_of(qt, kt, vt, mask, kv_count, out, lse, ws), stream,
         lambda s: load_library().bsa_sparse_attn_fwd(ctypes.byref(g.c()), _ptr(qt), _ptr(kt), _ptr(vt),
                                                      _ptr(mask), _ptr(kv_count), ctypes.c_float(sc),
                                                      _ptr(out), _ptr(lse), _ptr(ws),
                                                      ctypes.c_size_t(ws.numel()), s))
    return out, lse


def route_flags(g: Geometry, ws: torch.Tensor) -> torch.Tensor:
    """The route flags (uint8 [B, NQT], 1 = dense row) that build_mask left in `ws`: a view
    into the workspace, valid until the workspace is given to another build_mask."""
    _need_ws(ws)
    off = int(load_library().bsa_route_flags_offset(ctypes.byref(g.c())))
    if off == 0:
        raise ValueError("invalid geometry")
    return ws[off:off + g.B * g.NT].view(g.B, g.NT)


def sparse_attn_fwd_token(g: Geometry, qt: torch.Tensor, kt: torch.Tensor, vt: torch.Tensor,
                          mask: torch.Tensor, kv_count: torch.Tensor, dense: torch.Tensor,
                          token_radius: int, scale: float | None = None, out: torch.Tensor | None = None,
                          lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                          want_lse: bool = True, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Block-sparse attention under a token-level circular support of radius token_radius
    (tokens): local rows (dense == 0) see their window tiles token by token, as
    bsa_sparse_attn_fwd_token in include/bsa.h describes."""
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt)):
        _need(t, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), name)
    _need(mask, torch.int32, (g.B, g.H, g.NT, g.NW), "mask")
    _need(kv_count, torch.int32, (g.B, g.H, g.NT), "kv_count")
    _need(dense, torch.uint8, (g.B, g.NT), "dense")
    dev = qt.device
    if out is None:
        out = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, (g.B, g.N, g.H, g.d), "out")
    if want_lse and lse is None:
        lse = torch.empty((g.B, g.H, g.N), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, torch.float32, (g.B, g.H, g.N), "lse")
    if ws is None:
        ws = alloc_workspace(g, dev)
    _need_ws(ws)
    sc = 1.0 / math.sqrt(g.d) if scale is None else float(scale)
    _run("bsa_sparse_attn_fwd_token", _device_of(qt, kt, vt, mask, kv_count, dense, out, lse, ws), stream,
         lambda s: load_library().bsa_sparse_attn_fwd_token(
             ctypes.byref(g.c()), _ptr(qt), _ptr(kt), _ptr(vt), _ptr(mask), _ptr(kv_count), _ptr(dense),
             ctypes.c_int(int(token_radius)), ctypes.c_float(sc), _ptr(out), _ptr(lse), _ptr(ws),
             ctypes.c_size_t(ws.numel()), s))
    return out, lse


def sparse_attn_fwd_fixed_scratch(g: Geometry, qt: torch.Tensor, kt: torch.Tensor, vt: torch.Tensor,
                                  mask: torch.Tensor, kv_count: torch.Tensor,
                                  scale: float | None = None, out: torch.Tensor | None = None,
                                  lse: torch.Tensor | None = None,
                                  kernel_errors: torch.Tensor | None = None,
                                  want_lse: bool = True,
                                  stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Block-sparse attention whose scratch is the library's own fixed device array.

    For callers that cannot allocate device memory (a plug-in that receives tensors from a
    host application which owns all device memory, or a serving loop that forbids
    allocation after start-up): pass preallocated `out` / `lse` and nothing is allocated
    here or in the library. Limits and sharing rules are those of
    bsa_sparse_attn_fwd_fixed_scratch in include/bsa.h: one call at a time per device, and
    the first call on a device should come before any stream capture.
    `kernel_errors`, if given, is a 1-element int32 device tensor that receives the call's
    kernel error word.
    """
    for name, t in (("qt", qt), ("kt", kt), ("vt", vt)):
        _need(t, torch.bfloat16, (g.B, g.H, g.NT, 64, g.d), name)
    _need(mask, torch.int32, (g.B, g.H, g.NT, g.NW), "mask")
    _need(kv_count, torch.int32, (g.B, g.H, g.NT), "kv_count")
    dev = qt.device
    if out is None:
        out = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, (g.B, g.N, g.H, g.d), "out")
    if want_lse and lse is None:
        lse = torch.empty((g.B, g.H, g.N), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, torch.float32, (g.B, g.H, g.N), "lse")
    if kernel_errors is not None:
        _need(kernel_errors, torch.int32, (1,), "kernel_errors")
    sc = 1.0 / math.sqrt(g.d) if scale is None else float(scale)
    _run("bsa_sparse_attn_fwd_fixed_scratch", _device_of(qt, kt, vt, mask, kv_count, out, lse, kernel_errors),
         stream,
         lambda s: load_library().bsa_sparse_attn_fwd_fixed_scratch(
             ctypes.byref(g.c()), _ptr(qt), _ptr(kt), _ptr(vt), _ptr(mask), _ptr(kv_count),
             ctypes.c_float(sc), _ptr(out), _ptr(lse), _ptr(kernel_errors), s))
    return out, lse


def _owned_by(stream):
    """Allocations inside belong to `stream` (the current one if None): memory that only the
    call's own stream touches may then be freed, and reused there, as soon as the call returns."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """An output of a call on `stream`, whose memory belongs to it (see _owned_by)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _given(t: torch.Tensor | None, like: torch.Tensor, dtype, shape, name: str, stream) -> torch.Tensor:
    """The caller's output, checked, or a new one."""
    if t is None:
        return _new(like, shape, dtype, stream)
    _need(t, dtype, shape, name)
    return t


def cross_workspace_bytes(g: CrossGeometry) -> int:
    return int(load_library().bsa_cross_workspace_bytes(ctypes.byref(g.c())))


def alloc_cross_workspace(g: CrossGeometry, device=None) -> torch.Tensor:
    """A device workspace of cross_attn_fwd and cross_attn_bwd, its header (byte 0 = kernel error word)
    zeroed."""
    n = cross_workspace_bytes(g)
    if n == 0:
        raise ValueError("invalid geometry")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    ws[:256].zero_()
    return ws


def _need_strided(t: torch.Tensor, shape, name: str) -> None:
    """A bf16 tensor whose last axis is contiguous; the library checks the other strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last axis")


def _cross_inputs(g: CrossGeometry, q, k, v, kv_len, key_mask):
    """Checks them; a reference to their strides, or None where they are dense."""
    _need_strided(q, (g.B, g.N, g.H, g.d), "q")
    _need_strided(k, (g.B, g.M, g.Hkv, g.d), "k")
    _need_strided(v, (g.B, g.M, g.Hkv, g.d), "v")
    if kv_len is not None:
        _need(kv_len, torch.int32, (g.B,), "kv_len")
    if key_mask is not None:
        _need(key_mask, torch.bool, (g.B, g.M), "key_mask")
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        return None
    three = ctypes.c_longlong * 3
    return ctypes.byref(bsa_cross_strides(*(three(*t.stride()[:3]) for t in (q, k, v))))


def _cross_ws(g: CrossGeometry, ws, like: torch.Tensor, stream) -> torch.Tensor:
    if ws is None:
        with _owned_by(stream):
            return alloc_cross_workspace(g, like.device)
    _need_ws(ws)
    return ws


def cross_attn_fwd(g: CrossGeometry, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   kv_len: torch.Tensor | None = None, key_mask: torch.Tensor | None = None,
                   scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, want_lse: bool = True,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Attention of q [B,N,H,d] to the encoder's k, v [B,M,Hkv,d] (bf16; parts of a fused projection
    may be passed as they are, and k and v expanded over the items).

    kv_len (int32 [B]) and key_mask (bool [B,M]) say which keys of an item are valid; an item
    without one gives 0 and an lse of -inf. scale: finite, above 0. Outputs may not overlap inputs.
    Returns (out bf16 [B,N,H,d], lse fp32 [B,H,N])."""
    st = _cross_inputs(g, q, k, v, kv_len, key_mask)
    out = _given(out, q, torch.bfloat16, (g.B, g.N, g.H, g.d), "out", stream)
    if want_lse or lse is not None:
        lse = _given(lse, q, torch.float32, (g.B, g.H, g.N), "lse", stream)
    ws = _cross_ws(g, ws, q, stream)
    sc = 1.0 / math.sqrt(g.d) if scale is None else float(scale)
    _call("bsa_cross_attn_fwd", (q, k, v, kv_len, key_mask, out, lse, ws), stream, load_library().bsa_cross_attn_fwd,
          _cross_geom_ref(g), st, q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(kv_len), _addr(key_mask), sc,
          out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel())
    return out, lse


def cross_attn_bwd(g: CrossGeometry, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                   lse: torch.Tensor, dout: torch.Tensor, kv_len: torch.Tensor | None = None,
                   key_mask: torch.Tensor | None = None, scale: float | None = None,
                   dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of cross_attn_fwd from its inputs, its out and lse, and dout (contiguous): dq [B,N,H,d],
    and dk and dv [B,M,Hkv,d] per item, zero at keys that are not valid (all bf16). Outputs may not
    overlap inputs."""
    st = _cross_inputs(g, q, k, v, kv_len, key_mask)
    _need(out, torch.bfloat16, (g.B, g.N, g.H, g.d), "out")
    _need(dout, torch.bfloat16, (g.B, g.N, g.H, g.d), "dout")
    _need(lse, torch.float32, (g.B, g.H, g.N), "lse")
    dq = _given(dq, q, torch.bfloat16, (g.B, g.N, g.H, g.d), "dq", stream)
    dk = _given(dk, q, torch.bfloat16, (g.B, g.M, g.Hkv, g.d), "dk", stream)
    dv = _given(dv, q, torch.bfloat16, (g.B, g.M, g.Hkv, g.d), "dv", stream)
    ws = _cross_ws(g, ws, q, stream)
    sc = 1.0 / math.sqrt(g.d) if scale is None else float(scale)
    _call("bsa_cross_attn_bwd", (q, k, v, out, lse, dout, kv_len, key_mask, dq, dk, dv, ws), stream,
          load_library().bsa_cross_attn_bwd, _cross_geom_ref(g), st, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          out.data_ptr(), lse.data_ptr(), dout.data_ptr(), _addr(kv_len), _addr(key_mask), sc, dq.data_ptr(),
          dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), ws.numel())
    return dq, dk, dv


def _call(what: str, tensors, stream, fn, *args) -> None:
    """fn(*args, stream handle) on the one device of `tensors`, made current if it is not: _run for
    the calls whose few microseconds of marshalling count."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            _device_of(*tensors)
    if stream is None and dev.type == "cuda":
        handle = torch._C._cuda_getCurrentRawStream(dev.index)    # without the Stream object, 2 us
    else:
        handle = _stream(stream, dev).value or 0
    if torch.cuda.current_device() == dev.index:
        _check(fn(*args, handle), what)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, handle), what)


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=64)
def _cross_geom_ref(g: CrossGeometry):
    return ctypes.byref(g.c())


_NORM_TYPES = {torch.bfloat16: 0, torch.float32: 1}


@functools.lru_cache(maxsize=256)
def _norm_struct(*fields) -> bsa_norm_shape:
    return bsa_norm_shape(*fields)


def _norm_shape(x, y_dtype, weight, bias, eps, weight_offset) -> bsa_norm_shape:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dtype not in _NORM_TYPES or y_dtype not in _NORM_TYPES:
        raise ValueError(f"x and y must be bfloat16 or float32, got {x.dtype} and {y_dtype}")
    if x.dim() < 1 or x.numel() == 0 or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous [..., C] tensor with at least one row, got {tuple(x.shape)}")
    C = x.shape[-1]
    rows, xt, yt = x.numel() // C, _NORM_TYPES[x.dtype], _NORM_TYPES[y_dtype]
    if weight is None:
        if bias is not None:
            raise ValueError("a bias needs a weight of the same shape")
        return _norm_struct(rows, C, 1, 0, xt, yt, 1, float(eps), float(weight_offset))
    if not isinstance(weight, torch.Tensor) or weight.dtype not in _NORM_TYPES:
        raise ValueError("weight must be a bfloat16 or float32 tensor")
    shared, per_item = tuple(weight.shape) == (C,), x.dim() >= 2 and tuple(weight.shape) == (x.shape[0], C)
    if not shared and not per_item:
        raise ValueError(f"weight must have shape {(C,)}, or {(x.shape[0], C)} for one per batch item, "
                         f"got {tuple(weight.shape)}")
    _need(weight, weight.dtype, weight.shape, "weight")
    if bias is not None:
        _need(bias, weight.dtype, weight.shape, "bias")
    return _norm_struct(rows, C, 1 if shared else x.shape[0], 0 if shared else 1, xt, yt, _NORM_TYPES[weight.dtype],
                        float(eps), float(weight_offset))


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   eps: float = 1e-6, weight_offset: float = 0.0, out_dtype: torch.dtype | None = None,
                   y: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                   rstd: torch.Tensor | None = None, want_stats: bool = True,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor | None, torch.Tensor | None]:
    """Layer norm over the last axis of x [..., C] (bfloat16 or float32).

    weight, bias: absent, [C], or [x.shape[0], C] (one row per batch item, as the modulation of
    a diffusion transformer; weight_offset=1 where it is stored as the distance from one).
    y may be x itself where the types agree. Returns y (out_dtype, x's type unless given) and the fp32 mean and rstd of every row for
    the backward pass (None without want_stats)."""
    dt = y.dtype if y is not None and out_dtype is None else out_dtype or getattr(x, "dtype", None)
    f = _norm_shape(x, dt, weight, bias, eps, weight_offset)
    y = _given(y, x, dt, x.shape, "y", stream)
    if want_stats or mean is not None:
        mean = _given(mean, x, torch.float32, x.shape[:-1], "mean", stream)
    if want_stats or rstd is not None:
        rstd = _given(rstd, x, torch.float32, x.shape[:-1], "rstd", stream)
    _call("bsa_layer_norm_fwd", (x, weight, bias, y, mean, rstd), stream, load_library().bsa_layer_norm_fwd,
          ctypes.byref(f), x.data_ptr(), _addr(weight), _addr(bias), y.data_ptr(), _addr(mean), _addr(rstd))
    return y, mean, rstd


def layer_norm_workspace_bytes(x: torch.Tensor, weight: torch.Tensor | None = None) -> int:
    return int(load_library().bsa_layer_norm_workspace_bytes(
        ctypes.byref(_norm_shape(x, x.dtype, weight, None, 0.0, 0.0))))


def alloc_layer_norm_workspace(x: torch.Tensor, weight: torch.Tensor | None = None) -> torch.Tensor:
    """A workspace of layer_norm_bwd for rows like x's and a weight like this one."""
    n = layer_norm_workspace_bytes(x, weight)
    if n == 0:
        raise ValueError("invalid shape")
    return torch.empty(n, dtype=torch.uint8, device=x.device)


def layer_norm_bwd(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, weight_offset: float = 0.0, want_weight: bool = True,
                   want_bias: bool = True, dx: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                   dbias: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor | None, torch.Tensor | None]:
    """Gradients of layer_norm_fwd from x, dy (both contiguous) and its statistics: dx (x's type; may
    be x or dy itself where the types agree), and dweight and dbias in float32, of the weight's
    shape (None without a weight, or where they are not wanted)."""
    f = _norm_shape(x, getattr(dy, "dtype", None), weight, None, 0.0, weight_offset)
    _need(dy, dy.dtype, x.shape, "dy")
    _need(mean, torch.float32, x.shape[:-1], "mean")
    _need(rstd, torch.float32, x.shape[:-1], "rstd")
    if weight is None and (dweight is not None or dbias is not None):
        raise ValueError("dweight and dbias need the weight")
    want_weight = weight is not None and (want_weight or dweight is not None)
    want_bias = weight is not None and (want_bias or dbias is not None)
    dx = _given(dx, x, x.dtype, x.shape, "dx", stream)
    if want_weight:
        dweight = _given(dweight, x, torch.float32, weight.shape, "dweight", stream)
    if want_bias:
        dbias = _given(dbias, x, torch.float32, weight.shape, "dbias", stream)
    if ws is not None:
        _need_ws(ws)
    elif want_weight or want_bias:
        with _owned_by(stream):
            ws = alloc_layer_norm_workspace(x, weight)
    _call("bsa_layer_norm_bwd", (x, dy, mean, rstd, weight, dx, dweight, dbias, ws), stream,
          load_library().bsa_layer_norm_bwd, ctypes.byref(f), x.data_ptr(), dy.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), _addr(weight), dx.data_ptr(), _addr(dweight), _addr(dbias), _addr(ws),
          0 if ws is None else ws.numel())
    return dx, dweight, dbias


class Buffers:
    """Device buffers of one attention call, allocated once and reused across calls."""

    def __init__(self, g: Geometry, device=None):
        dev = device or "cuda"
        tiled = (g.B, g.H, g.NT, 64, g.d)
        self.qt = torch.empty(tiled, dtype=torch.bfloat16, device=dev)
        self.kt = torch.empty(tiled, dtype=torch.bfloat16, device=dev)
        self.vt = torch.empty(tiled, dtype=torch.bfloat16, device=dev)
        self.qbar = torch.empty((g.B, g.H, g.NT, g.d), dtype=torch.float32, device=dev)
        self.kbar = torch.empty((g.B, g.H, g.NT, g.d), dtype=torch.float32, device=dev)
        self.mask = torch.empty((g.B, g.H, g.NT, g.NW), dtype=torch.int32, device=dev)
        self.kv_count = torch.empty((g.B, g.H, g.NT), dtype=torch.int32, device=dev)
        self.out = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((g.B, g.H, g.N), dtype=torch.float32, device=dev)
        self.ws = alloc_workspace(g, dev)


@dataclass(frozen=True)
class QKNorm:
    """Layer norm of Q and K over the head dimension ahead of attention: weights and biases [d]
    (bfloat16 or float32), shared by all heads and tokens; None for none. Models that normalise Q
    and K by their root mean square need a norm of their own ahead of the call."""

    q_weight: torch.Tensor | None = None
    q_bias: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    k_bias: torch.Tensor | None = None
    eps: float = 1e-6


class CrossBuffers:
    """Device buffers of one cross_forward call, allocated once and reused across calls."""

    def __init__(self, g: CrossGeometry, qk_norm: bool = False, device=None):
        dev = device or "cuda"
        self.qn = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=dev) if qk_norm else None
        self.kn = torch.empty((g.B, g.M, g.Hkv, g.d), dtype=torch.bfloat16, device=dev) if qk_norm else None
        self.out = torch.empty((g.B, g.N, g.H, g.d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((g.B, g.H, g.N), dtype=torch.float32, device=dev)
        self.ws = alloc_cross_workspace(g, dev)


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two contiguous tensors share memory."""
    lo, hi = a.data_ptr(), b.data_ptr()
    return lo < hi + b.numel() * b.element_size() and hi < lo + a.numel() * a.element_size()


def cross_forward(g: CrossGeometry, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  kv_len: torch.Tensor | None = None, key_mask: torch.Tensor | None = None,
                  qk_norm: QKNorm | None = None, bufs: CrossBuffers | None = None, scale: float | None = None,
                  stream=None) -> CrossBuffers:
    """The attention to an encoder's states as a block runs it: the norm of Q and K per head, if
    any (q and k are then contiguous), and cross_attn_fwd. Returns the buffers; out and lse hold
    the result. The way back is made of cross_attn_bwd on qn and kn and of layer_norm_bwd, for which
    layer_norm_fwd gives the statistics of q and k."""
    if bufs is None:
        with _owned_by(stream):
            bufs = CrossBuffers(g, qk_norm is not None, q.device)
    if qk_norm is not None:
        if bufs.qn is None:
            raise ValueError("these buffers have no room for the norm: CrossBuffers(g, qk_norm=True)")
        n = qk_norm
        layer_norm_fwd(q, n.q_weight, n.q_bias, n.eps, y=bufs.qn, want_stats=False, stream=stream)
        layer_norm_fwd(k, n.k_weight, n.k_bias, n.eps, y=bufs.kn, want_stats=False, stream=stream)
        q, k = bufs.qn, bufs.kn
    cross_attn_fwd(g, q, k, v, kv_len, key_mask, scale, bufs.out, bufs.lse, bufs.ws, stream=stream)
    return bufs


def forward(g: Geometry, p: MaskParams, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
            difficulty: torch.Tensor, bufs: Buffers | None = None, scale: float | None = None,
            stream=None, rebuild_mask: bool = True, qk_norm: QKNorm | None = None) -> Buffers:
    """The whole path: reorder Q, K, V; build the mask; block-sparse attention.

    Returns the buffers; out / lse hold the attention output and LSE in raster order.
    rebuild_mask=False skips the mask build and attends through the mask (and counts) that
    an earlier call left in `bufs`: the reuse of a previous step's routing and sparsity
    (HetA-DiT reuses the preceding denoising step's estimates; MOD-DiT keeps historical
    sparsity). How often to rebuild is the caller's choice.
    With window kind 2 (token-level circular support, radius p.radius in tokens) the
    attention masks the tokens outside each query token's support inside window tiles,
    with the route flags the mask build left in the workspace.
    qk_norm: layer norm of Q and K over the head dimension first (the mask is then that of the
    normalised Q and K). q, k and v may be the `out` of an earlier call on these buffers.
    """
    if not rebuild_mask and bufs is None:
        raise ValueError("rebuild_mask=False attends through the mask held in bufs: pass the "
                         "Buffers of an earlier call")
    b = bufs or Buffers(g, q.device)
    # The normalised Q and K pass through `out`, which is not written before V has been reordered; or,
    # where an input lies there, through the tile-major buffer that is filled next.
    taken = False
    if qk_norm is not None:
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            _need(t, torch.bfloat16, (g.B, g.N, g.H, g.d), name)
            taken |= _overlap(t, b.out)
    for x, xt, xbar, norm, free in ((q, b.qt, b.qbar, qk_norm and (qk_norm.q_weight, qk_norm.q_bias), b.kt),
                                    (k, b.kt, b.kbar, qk_norm and (qk_norm.k_weight, qk_norm.k_bias), b.vt)):
        if qk_norm is not None:
            y = free.view(-1)[:x.numel()].view(x.shape) if taken else b.out
            x, _, _ = layer_norm_fwd(x, *norm, qk_norm.eps, y=y, want_stats=False, stream=stream)
        if rebuild_mask:
            reorder_pool(g, x, xt, xbar, stream)
        else:
            reorder(g, x, xt, stream)
    reorder(g, v, b.vt, stream)
    if rebuild_mask:
        build_mask_pooled(g, p, b.qbar, b.kbar, difficulty, b.mask, b.kv_count, b.ws, stream)
    if p.window_kind == 2:
        sparse_attn_fwd_token(g, b.qt, b.kt, b.vt, b.mask, b.kv_count, route_flags(g, b.ws), p.radius,
                              scale, b.out, b.lse, b.ws, stream=stream)
    else:
        sparse_attn_fwd(g, b.qt, b.kt, b.vt, b.mask, b.kv_count, scale, b.out, b.lse, b.ws,
                        stream=stream)
    return b


# kernels launched by forward(): 3 reorders (Q and K fused with their pooling when the
# mask is rebuilt); route, score and select (plus entropy and budget in budget mode) unless
# the mask is reused; 3 scheduler kernels and the attention kernel; 2 norms with qk_norm
def launches_per_forward(p: MaskParams, rebuild_mask: bool = True, qk_norm: bool = False) -> int:
    return 3 + ((3 + (2 if p.budget_mode == 1 else 0)) if rebuild_mask else 0) + 4 + (2 if qk_norm else 0)
