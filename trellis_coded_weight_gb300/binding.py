"""Thin ctypes binding of libtrellis.so (the C ABI in include/trellis.h).

Argument marshalling only: each function checks the tensors' device, dtype,
shape and contiguity, passes raw device pointers and the current CUDA stream
to the C entry point of the same name, and raises on a non-zero status.  Every
step of the computation runs in the library's CUDA kernels; there is no
fallback -- if the library cannot be loaded, every call raises.

bf16 tensors are torch.bfloat16; fp16 scales are torch.float16; codes are
torch.int32 or torch.uint32 tensors holding the packed words.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from dataclasses import dataclass
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtrellis.so")

TRELLIS_OK = 0
STATUS_NAMES = {0: "TRELLIS_OK", -1: "TRELLIS_EGEOM", -2: "TRELLIS_EM", -3: "TRELLIS_EALIGN", -4: "TRELLIS_EAXIS",
                -5: "TRELLIS_EWORKSPACE", -6: "TRELLIS_ECUDA", -7: "TRELLIS_ENULL", -8: "TRELLIS_EDEVICE",
                -9: "TRELLIS_ESHAPE"}

EXPORTS = ("trellis_abi_version", "trellis_status_string", "trellis_check_geom", "trellis_expand_bf16",
           "trellis_matvec_axis1", "trellis_matvec_axis0", "trellis_workspace_bytes", "trellis_gateup_swiglu",
           "trellis_gemm_prefill", "trellis_device_error", "trellis_mlp_decode", "trellis_matvec_axis1_bf16w",
           "trellis_matvec_axis0_bf16w", "trellis_load_floor", "trellis_load_floor_rows", "trellis_prefill_plan",
           "trellis_set_wait_limit", "trellis_matvec_axis1_host", "trellis_check_cache", "trellis_qk_norm_rope_append",
           "trellis_tree_attention", "trellis_tree_workspace_bytes", "trellis_cache_copy", "trellis_cache_fork",
           "trellis_cache_compact", "trellis_cache_workspace_bytes", "trellis_cache_commit", "trellis_token_logprobs",
           "trellis_logprobs_workspace_bytes")


class TrellisGeom(ctypes.Structure):
    """Mirror of trellis_geom_t."""
    _fields_ = [("k", ctypes.c_int32), ("L", ctypes.c_int32), ("T", ctypes.c_int32), ("axis", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("interleave", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


@dataclass(frozen=True)
class Geometry:
    """Stored-matrix geometry: k bits/weight, L-bit windows, T-long blocks."""
    k: int
    L: int
    T: int
    axis: int
    rows: int
    cols: int
    interleave: int = 0  # 2: the k=3 axis-0 layout [cols/512][rows][48]

    def c(self) -> TrellisGeom:
        """The C struct of this geometry (built once per geometry and kept)."""
        g = _GEOM_STRUCTS.get(self)
        if g is None:
            g = _GEOM_STRUCTS.setdefault(self, TrellisGeom(self.k, self.L, self.T, self.axis, self.rows, self.cols,
                                                           self.interleave, 0))
        return g

    @property
    def words_per_row(self) -> int:
        return self.cols * self.k // 32

    @property
    def codes_shape(self) -> tuple:
        if self.interleave:
            return (self.cols // (2 * self.T), self.rows, 2 * self.T * self.k // 32)
        return (self.rows, self.words_per_row)


_GEOM_STRUCTS: dict = {}


class TrellisError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({msg})")
        self.status = status


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libtrellis.so (raises if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libtrellis.so not built at {path}; run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            g = ctypes.POINTER(TrellisGeom)
            lib.trellis_abi_version.restype = i32
            lib.trellis_abi_version.argtypes = []
            lib.trellis_status_string.restype = ctypes.c_char_p
            lib.trellis_status_string.argtypes = [i32]
            lib.trellis_check_geom.restype = i32
            lib.trellis_check_geom.argtypes = [g]
            lib.trellis_expand_bf16.restype = i32
            lib.trellis_expand_bf16.argtypes = [vp, vp, vp, g, vp]
            lib.trellis_matvec_axis1.restype = i32
            lib.trellis_matvec_axis1.argtypes = [vp, vp, vp, vp, i32, g, vp]
            lib.trellis_matvec_axis0.restype = i32
            lib.trellis_matvec_axis0.argtypes = [vp, vp, vp, vp, i32, g, vp, sz, vp]
            lib.trellis_workspace_bytes.restype = sz
            lib.trellis_workspace_bytes.argtypes = [i32, g]
            lib.trellis_gateup_swiglu.restype = i32
            lib.trellis_gateup_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, i32, g, vp]
            lib.trellis_gemm_prefill.restype = i32
            lib.trellis_gemm_prefill.argtypes = [vp, vp, vp, vp, i32, g, vp]
            lib.trellis_matvec_axis1_host.restype = i32
            lib.trellis_matvec_axis1_host.argtypes = [vp, vp, vp, vp, i32, g, vp, vp, vp]
            lib.trellis_matvec_axis1_bf16w.restype = i32
            lib.trellis_matvec_axis1_bf16w.argtypes = [vp, vp, vp, vp, i32, g, vp]
            lib.trellis_matvec_axis0_bf16w.restype = i32
            lib.trellis_matvec_axis0_bf16w.argtypes = [vp, vp, vp, vp, i32, g, vp, sz, vp]
            lib.trellis_mlp_decode.restype = i32
            lib.trellis_mlp_decode.argtypes = [vp] * 9 + [i32, g, g, vp, sz, vp]
            lib.trellis_device_error.restype = i32
            lib.trellis_device_error.argtypes = [i32]
            lib.trellis_set_wait_limit.restype = i32
            lib.trellis_set_wait_limit.argtypes = [ctypes.c_uint64]
            lib.trellis_load_floor.restype = i32
            lib.trellis_load_floor.argtypes = [vp, vp, g, vp]
            lib.trellis_load_floor_rows.restype = i32
            lib.trellis_load_floor_rows.argtypes = [vp, vp, g, vp]
            lib.trellis_prefill_plan.restype = i32
            lib.trellis_prefill_plan.argtypes = [i32, g, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
            _lib = lib
    return _lib


def _check(fn: str, status: int):
    if status != TRELLIS_OK:
        raise TrellisError(fn, status, load().trellis_status_string(status).decode())


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _on(t: torch.Tensor):
    """Make the tensor's device current for the C call: the library reads the
    current device (its SM count, kernel attributes) and launches on it."""
    if t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _req(t: torch.Tensor, name: str, dtypes, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_CODES = (torch.int32, getattr(torch, "uint32", torch.int32))


def expand_bf16(codes, scales, g: Geometry, out=None):
    """Decoded stored matrix [rows, cols] bf16 (bit-exact)."""
    if out is None:
        out = torch.empty((g.rows, g.cols), dtype=torch.bfloat16, device=codes.device)
    args = (_req(codes, "codes", _CODES, g.codes_shape),
            _req(scales, "scales", (torch.float16,), (g.rows,)),
            _req(out, "out", (torch.bfloat16,), (g.rows, g.cols)))
    with _on(codes):
        _check("trellis_expand_bf16", load().trellis_expand_bf16(*args, ctypes.byref(g.c()), _stream(codes)))
    return out


def matvec_axis1(codes, scales, x, g: Geometry, out=None, bf16_weights: bool = False):
    """out[M, rows] = x[M, cols] @ W^T for an axis-1 matrix, M = 1..4.

    bf16_weights selects the bf16-rounded weight numerics (the expand weights)."""
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, g.rows), dtype=torch.bfloat16, device=x.device)
    args = (_req(codes, "codes", _CODES, g.codes_shape),
            _req(scales, "scales", (torch.float16,), (g.rows,)),
            _req(x, "x", (torch.bfloat16,), (M, g.cols)),
            _req(out, "out", (torch.bfloat16,), (M, g.rows)))
    fn = "trellis_matvec_axis1_bf16w" if bf16_weights else "trellis_matvec_axis1"
    with _on(x):
        _check(fn, getattr(load(), fn)(*args, M, ctypes.byref(g.c()), _stream(x)))
    return out


def _req_host(t: torch.Tensor, name: str, shape):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def matvec_axis1_host(codes, scales, x_host, g: Geometry, out_host, x_dev, out_dev):
    """matvec_axis1 with x and out on the host: one C call queues x_host -> x_dev, the matvec and its output's
    transfer to out_host on the current stream of the codes' device.  out_host holds the result once that stream
    has reached the call (synchronize before reading it).  Pinned (16-byte aligned) host tensors are reached
    through their device mapping: a copy kernel fills x_dev and the matvec writes out_host directly, leaving
    out_dev untouched; other host tensors go through copy-engine copies via x_dev and out_dev."""
    M = x_host.shape[0]
    args = (_req(codes, "codes", _CODES, g.codes_shape),
            _req(scales, "scales", (torch.float16,), (g.rows,)),
            _req_host(x_host, "x_host", (M, g.cols)),
            _req_host(out_host, "out_host", (M, g.rows)))
    xd = _req(x_dev, "x_dev", (torch.bfloat16,), (M, g.cols))
    od = _req(out_dev, "out_dev", (torch.bfloat16,), (M, g.rows))
    with _on(codes):
        _check("trellis_matvec_axis1_host",
               load().trellis_matvec_axis1_host(*args, M, ctypes.byref(g.c()), xd, od, _stream(codes)))
    return out_host


def workspace_bytes(M: int, g: Geometry) -> int:
    return int(load().trellis_workspace_bytes(M, ctypes.byref(g.c())))


def new_workspace(M: int, g: Geometry, device) -> torch.Tensor:
    """A zero-filled workspace for matvec_axis0 (reusable across calls)."""
    n = workspace_bytes(M, g)
    if n == 0:
        raise ValueError("unsupported geometry or M for the axis-0 matvec")
    return torch.zeros(((n + 15) // 16) * 4, dtype=torch.int32, device=device)


def matvec_axis0(codes, scales, x, g: Geometry, workspace, out=None, bf16_weights: bool = False):
    """out[M, cols] = x[M, rows] @ W^T for an axis-0 matrix (stored W^T), M = 1..4.

    bf16_weights selects the bf16-rounded weight numerics (the expand weights)."""
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, g.cols), dtype=torch.bfloat16, device=x.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    args = (_req(codes, "codes", _CODES, g.codes_shape),
            _req(scales, "scales", (torch.float16,), (g.rows,)),
            _req(x, "x", (torch.bfloat16,), (M, g.rows)),
            _req(out, "out", (torch.bfloat16,), (M, g.cols)))
    nbytes = workspace.numel() * workspace.element_size()
    fn = "trellis_matvec_axis0_bf16w" if bf16_weights else "trellis_matvec_axis0"
    with _on(x):
        _check(fn, getattr(load(), fn)(*args, M, ctypes.byref(g.c()), workspace.data_ptr(), nbytes, _stream(x)))
    return out


def gateup_swiglu(gcodes, gscales, ucodes, uscales, x, g: Geometry, out=None):
    """out[M, rows] = bf16 SwiGLU chain of the gate and up matvecs, M = 1..4."""
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, g.rows), dtype=torch.bfloat16, device=x.device)
    shp = g.codes_shape
    args = (_req(gcodes, "gcodes", _CODES, shp), _req(gscales, "gscales", (torch.float16,), (g.rows,)),
            _req(ucodes, "ucodes", _CODES, shp), _req(uscales, "uscales", (torch.float16,), (g.rows,)),
            _req(x, "x", (torch.bfloat16,), (M, g.cols)), _req(out, "out", (torch.bfloat16,), (M, g.rows)))
    with _on(x):
        _check("trellis_gateup_swiglu", load().trellis_gateup_swiglu(*args, M, ctypes.byref(g.c()), _stream(x)))
    return out


def gemm_prefill(codes, scales, x, g: Geometry, out=None):
    """Prefill GEMM on the tensor cores with the bf16 expand weights E (stored [rows, cols]):
    axis 1: out[M, rows] = x[M, cols] @ E^T;  axis 0: out[M, cols] = x[M, rows] @ E."""
    M = x.shape[0]
    n_in, n_out = (g.cols, g.rows) if g.axis == 1 else (g.rows, g.cols)
    if out is None:
        out = torch.empty((M, n_out), dtype=torch.bfloat16, device=x.device)
    args = (_req(codes, "codes", _CODES, g.codes_shape),
            _req(scales, "scales", (torch.float16,), (g.rows,)),
            _req(x, "x", (torch.bfloat16,), (M, n_in)),
            _req(out, "out", (torch.bfloat16,), (M, n_out)))
    with _on(x):
        _check("trellis_gemm_prefill", load().trellis_gemm_prefill(*args, M, ctypes.byref(g.c()), _stream(x)))
    return out


def load_floor(codes: torch.Tensor, g: Geometry, out: torch.Tensor = None, coalesced: bool = False) -> torch.Tensor:
    """Measurement aid: read the axis-1 stream and decode nothing; out[r] = XOR of the words loaded for row r
    (int32 view of uint32).  Default: the M = 1 matvec's access pattern (lane per row); coalesced: a warp per
    row with its lanes on consecutive 16-byte chunks."""
    if out is None:
        out = torch.empty(g.rows, dtype=torch.int32, device=codes.device)
    args = (_req(codes, "codes", _CODES, g.codes_shape), _req(out, "out", (torch.int32,), (g.rows,)))
    fn = "trellis_load_floor_rows" if coalesced else "trellis_load_floor"
    with _on(codes):
        _check(fn, getattr(load(), fn)(*args, ctypes.byref(g.c()), _stream(codes)))
    return out


def prefill_plan(M: int, g: Geometry, sms: int = 0):
    """The tile plan of gemm_prefill (host arithmetic): (tokens per tile, [(first tile, tiles, CTAs per
    tile), ...]).  sms < 1 takes the current device's SM count."""
    bn = ctypes.c_int32(0)
    buf = (ctypes.c_int32 * 6)()
    n = load().trellis_prefill_plan(M, ctypes.byref(g.c()), sms, ctypes.byref(bn), buf)
    _check("trellis_prefill_plan", n if n < 0 else 0)
    return bn.value, [tuple(buf[3 * i:3 * i + 3]) for i in range(n)]


def set_wait_limit(nanoseconds: int = 0) -> None:
    """Diagnostic: limit of each bounded wait of the tensor-core kernel for later launches (0: the default)."""
    _check("trellis_set_wait_limit", load().trellis_set_wait_limit(int(nanoseconds)))


def device_error(reset: bool = False) -> int:
    """Device error word of the tensor-core kernel (0 = no bounded wait gave up)."""
    return int(load().trellis_device_error(1 if reset else 0))


def mlp_decode(gcodes, gscales, ucodes, uscales, dcodes, dscales, x, g_up: Geometry, g_down: Geometry, workspace,
               hidden=None, out=None):
    """Decode-time MLP block: out = down(swiglu(gate(x), up(x))), M = 1..4 (two launches)."""
    M = x.shape[0]
    if hidden is None:
        hidden = torch.empty((M, g_up.rows), dtype=torch.bfloat16, device=x.device)
    if out is None:
        out = torch.empty((M, g_down.cols), dtype=torch.bfloat16, device=x.device)
    shp_u, shp_d = g_up.codes_shape, g_down.codes_shape
    args = (_req(gcodes, "gcodes", _CODES, shp_u), _req(gscales, "gscales", (torch.float16,), (g_up.rows,)),
            _req(ucodes, "ucodes", _CODES, shp_u), _req(uscales, "uscales", (torch.float16,), (g_up.rows,)),
            _req(dcodes, "dcodes", _CODES, shp_d), _req(dscales, "dscales", (torch.float16,), (g_down.rows,)),
            _req(x, "x", (torch.bfloat16,), (M, g_up.cols)), _req(hidden, "hidden", (torch.bfloat16,), (M, g_up.rows)),
            _req(out, "out", (torch.bfloat16,), (M, g_down.cols)))
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    nbytes = workspace.numel() * workspace.element_size()
    with _on(x):
        _check("trellis_mlp_decode", load().trellis_mlp_decode(*args, M, ctypes.byref(g_up.c()),
                                                              ctypes.byref(g_down.c()), workspace.data_ptr(), nbytes,
                                                              _stream(x)))
    return hidden, out


class MlpDecodeGraph:
    """The decode MLP block captured once into a CUDA graph and replayed.

    Buffers (x, hidden, out, workspace) are fixed at capture time; write the
    next token's activations into `x` and call `replay()`.
    """

    def __init__(self, gcodes, gscales, ucodes, uscales, dcodes, dscales, g_up: Geometry, g_down: Geometry, M: int):
        dev = gcodes.device
        self.x = torch.zeros((M, g_up.cols), dtype=torch.bfloat16, device=dev)
        self.hidden = torch.empty((M, g_up.rows), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((M, g_down.cols), dtype=torch.bfloat16, device=dev)
        self.workspace = new_workspace(M, g_down, dev)
        self._args = (gcodes, gscales, ucodes, uscales, dcodes, dscales)
        self._g = (g_up, g_down)
        s = torch.cuda.Stream(device=dev)
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):  # warm-up launch outside the graph (library set-up, first-use costs)
            mlp_decode(*self._args, self.x, *self._g, self.workspace, self.hidden, self.out)
        torch.cuda.current_stream(dev).wait_stream(s)
        torch.cuda.synchronize(dev)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            mlp_decode(*self._args, self.x, *self._g, self.workspace, self.hidden, self.out)

    def replay(self):
        self.graph.replay()
        return self.out


# ---- The rest of a decoding step: paged cache, norms with rotation, tree attention, token log probabilities ----

TRELLIS_BF16, TRELLIS_E4M3, TRELLIS_F32 = 0, 1, 2


class TrellisCache(ctypes.Structure):
    """Mirror of trellis_cache_t."""
    _fields_ = [("pool", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("layers", ctypes.c_int32), ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class TrellisNormRope(ctypes.Structure):
    """Mirror of trellis_norm_rope_t."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("max_pos", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class TrellisDrafts(ctypes.Structure):
    """Mirror of trellis_drafts_t."""
    _fields_ = [("table", ctypes.c_void_p), ("prefix", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("batch", ctypes.c_int32), ("width", ctypes.c_int32), ("n", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32)]


_BF16, _I32, _I64, _FP32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
_current_device = torch._C._cuda_getDevice
_stream_of_index = torch._C._cuda_getCurrentRawStream


def _raw_stream(device: torch.device) -> int:
    return _stream_of_index(device.index)


def _call(fn: str, index: int, *args):
    """The C call of that name with device `index` current and its current stream as the last argument.

    The calls of a decoding step are a few microseconds on the GPU, so the functions below test all arguments in one
    expression first and only go through the messages of _req_tokens and _req_rows when it fails."""
    f = getattr(_serving_lib(), fn)
    if _current_device() == index:
        st = f(*args, _stream_of_index(index))
    else:
        with torch.cuda.device(index):
            st = f(*args, _stream_of_index(index))
    if st:
        _check(fn, st)


def _same_device(device: torch.device, **tensors):
    for name, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _req_tokens(t: torch.Tensor, name: str, n: int, heads: int, dim: int):
    """A bf16 [n, heads, dim] tensor whose tokens may be apart (a slice of a wider projection): pointer, stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    if t.shape != (n, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n, heads, dim)}")
    stride, per_head, one = t.stride()
    if (one != 1 and dim > 1) or (per_head != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), stride


def _req_rows(t: torch.Tensor, name: str, dtype, shape):
    """As _req for one dtype."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _req_workspace(t: torch.Tensor):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return t.data_ptr(), t.numel() * t.element_size()


_serving = None


def _serving_lib():
    """The library with the argument types of the serving calls set (once)."""
    global _serving
    if _serving is None:
        lib = load()
        vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        cache = ctypes.POINTER(TrellisCache)
        for name, res, args in (
                ("trellis_check_cache", i32, [cache]),
                ("trellis_qk_norm_rope_append", i32, [vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, i32,
                                                      ctypes.POINTER(TrellisNormRope), cache, i32, vp]),
                ("trellis_tree_attention", i32, [vp, i64, cache, i32, ctypes.POINTER(TrellisDrafts), i32, f32, vp, i64,
                                                 vp, vp, sz, vp]),
                ("trellis_tree_workspace_bytes", sz, [cache, i32, i32, i32]),
                ("trellis_cache_copy", i32, [cache, vp, vp, i32, vp]),
                ("trellis_cache_fork", i32, [cache, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, sz, vp]),
                ("trellis_cache_compact", i32, [cache, vp, vp, vp, vp, i32, i32, vp, sz, vp]),
                ("trellis_cache_workspace_bytes", sz, [cache, i32, i32]),
                ("trellis_cache_commit", i32, [cache, vp, vp, vp, vp, vp, i32, i32, i32, vp]),
                ("trellis_token_logprobs", i32, [vp, i32, i64, vp, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, sz,
                                                 vp]),
                ("trellis_logprobs_workspace_bytes", sz, [i32, i32, i32])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _serving = lib
    return _serving


class PagedCache:
    """A paged key/value cache of all layers: pool [layers, pages, 2, heads, page_size, head_dim], bf16 or e4m3
    (torch.float8_e4m3fn, with scales [layers, 2, heads] fp32 or None for ones).  Keeps the tensors it describes."""

    def __init__(self, pool: torch.Tensor, scales: torch.Tensor = None):
        if not isinstance(pool, torch.Tensor) or not pool.is_cuda:
            raise ValueError("pool must be a CUDA tensor")
        if pool.dim() != 6 or pool.shape[2] != 2:
            raise ValueError(f"pool has shape {tuple(pool.shape)}, expected [layers, pages, 2, heads, page_size, head_dim]")
        if pool.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"pool has dtype {pool.dtype}, expected torch.bfloat16 or torch.float8_e4m3fn")
        if not pool.is_contiguous():
            raise ValueError("pool must be contiguous")
        self.pool, self.scales, self.device, self.index = pool, scales, pool.device, pool.get_device()
        self.layers, self.pages, _, self.heads, self.page_size, self.head_dim = pool.shape
        if scales is not None:
            if pool.dtype != torch.float8_e4m3fn:
                raise ValueError("scales belong to an e4m3 pool")
            _req_rows(scales, "scales", torch.float32, (self.layers, 2, self.heads))
            _same_device(self.device, scales=scales)
        self._c = TrellisCache(pool.data_ptr(), scales.data_ptr() if scales is not None else None, self.pages, self.layers,
                               self.heads, self.page_size, self.head_dim,
                               TRELLIS_E4M3 if pool.dtype == torch.float8_e4m3fn else TRELLIS_BF16, 0)
        self._ref = ctypes.byref(self._c)
        _check("trellis_check_cache", _serving_lib().trellis_check_cache(self._ref))

    @classmethod
    def new(cls, layers, pages, heads, page_size, head_dim, device, dtype=torch.bfloat16, scales=None):
        """A cache over a fresh (zeroed) pool."""
        return cls(torch.zeros((layers, pages, 2, heads, page_size, head_dim), dtype=dtype, device=device), scales)


class NormRope:
    """The weights, rotation table and constants of a layer's query/key norms (trellis_norm_rope_t).

    rope [max_pos, rotary_dim] fp32: rotary_dim/2 cosines, then as many sines, per position; None: no rotation.
    interleaved pairs dim 2i with 2i + 1, else i with i + rotary_dim/2."""

    def __init__(self, q_weight, k_weight, rope, q_heads: int, kv_heads: int, interleaved: bool = False, eps: float = 1e-6,
                 weight_offset: float = 0.0):
        dim = q_weight.shape[-1]
        _req_rows(q_weight, "q_weight", torch.bfloat16, (dim,))
        _req_rows(k_weight, "k_weight", torch.bfloat16, (dim,))
        _same_device(q_weight.device, k_weight=k_weight)
        if rope is not None:
            _req_rows(rope, "rope", torch.float32, (rope.shape[0], rope.shape[-1]))
            _same_device(q_weight.device, rope=rope)
        self.q_heads, self.kv_heads, self.head_dim, self.device = q_heads, kv_heads, dim, q_weight.device
        self.index = q_weight.get_device()
        self._kept = (q_weight, k_weight, rope)
        # without rotation there is no table, and any position is in range
        self._c = TrellisNormRope(q_weight.data_ptr(), k_weight.data_ptr(), rope.data_ptr() if rope is not None else None,
                                  rope.shape[0] if rope is not None else 1 << 31, q_heads, kv_heads, dim,
                                  rope.shape[1] if rope is not None else 0, int(interleaved), 0, eps, weight_offset)
        self._ref = ctypes.byref(self._c)


def qk_norm_rope_append(q, k, v, positions, slots, norm: NormRope, cache: PagedCache, layer: int, out=None):
    """Per-head norms of q [n, q_heads, dim] and k [n, kv_heads, dim], the rotation by positions [n] int32, and the
    write of k and v to slots [n] int64 (page * page_size + row; negative: none) of the cache's layer, in one launch.
    q, k and v may be slices of one projection.  Returns the queries (out may be q)."""
    n, dim, index = q.shape[0], norm.head_dim, cache.index
    if out is None:
        out = torch.empty((n, norm.q_heads, dim), dtype=_BF16, device=cache.device)
    wide, narrow, row, inner = (n, norm.q_heads, dim), (n, norm.kv_heads, dim), (n,), (dim, 1)
    qs, ks, vs, os_ = q.stride(), k.stride(), v.stride(), out.stride()
    if not (q.dtype is _BF16 and k.dtype is _BF16 and v.dtype is _BF16 and out.dtype is _BF16 and positions.dtype is _I32 and
            slots.dtype is _I64 and q.shape == wide and out.shape == wide and k.shape == narrow and v.shape == narrow and
            positions.shape == row and slots.shape == row and qs[1:] == inner and ks[1:] == inner and vs[1:] == inner and
            os_[1:] == inner and positions.is_contiguous() and slots.is_contiguous() and
            q.get_device() == k.get_device() == v.get_device() == out.get_device() == positions.get_device() ==
            slots.get_device() == norm.index == index):
        for t, name, shape in ((q, "q", wide), (k, "k", narrow), (v, "v", narrow), (out, "out", wide)):
            _req_tokens(t, name, *shape)
        _req_rows(positions, "positions", _I32, row)
        _req_rows(slots, "slots", _I64, row)
        _same_device(cache.device, q=q, k=k, v=v, out=out, positions=positions, slots=slots, norm=norm)
    _call("trellis_qk_norm_rope_append", index, q.data_ptr(), qs[0], k.data_ptr(), ks[0], v.data_ptr(), vs[0],
          positions.data_ptr(), slots.data_ptr(), out.data_ptr(), os_[0], n, norm._ref, cache._ref, layer)
    return out


class DraftBatch:
    """One step's sequences and drafted tokens (trellis_drafts_t), shared by the step's layers.

    table [batch, width] int32 pages;  prefix [batch] int32 positions before the drafts;  q_start [batch + 1] int32
    (sequence b's drafts are tokens q_start[b] .. q_start[b+1] - 1);  max_tokens: most drafts of a sequence (<= 64);
    mask [n] int64: bit j set where the token sees draft j of its sequence (None: drafts 0 .. itself, then n is
    needed).  Keeps the tensors; their contents are read by each call."""

    def __init__(self, table, prefix, q_start, max_tokens: int, mask=None, n: int = None):
        batch, width = table.shape
        if mask is not None:
            n = mask.shape[0] if n is None else n
            _req_rows(mask, "mask", torch.int64, (n,))
        elif n is None:
            raise ValueError("n is needed without a mask")
        _req_rows(table, "table", torch.int32, (batch, width))
        _req_rows(prefix, "prefix", torch.int32, (batch,))
        _req_rows(q_start, "q_start", torch.int32, (batch + 1,))
        _same_device(table.device, prefix=prefix, q_start=q_start, **({} if mask is None else {"mask": mask}))
        self.table, self.prefix, self.q_start, self.mask = table, prefix, q_start, mask
        self.batch, self.width, self.n, self.max_tokens, self.device = batch, width, n, max_tokens, table.device
        self.index = table.get_device()
        self._c = TrellisDrafts(table.data_ptr(), prefix.data_ptr(), q_start.data_ptr(),
                                mask.data_ptr() if mask is not None else None, batch, width, n, max_tokens)
        self._ref = ctypes.byref(self._c)


def _workspace(nbytes: int, device, what: str) -> torch.Tensor:
    if nbytes == 0:
        raise ValueError(f"unsupported sizes for {what}")
    return torch.zeros((nbytes + 15) // 16 * 4, dtype=torch.int32, device=device)


def new_tree_workspace(cache: PagedCache, batch: DraftBatch, q_heads: int) -> torch.Tensor:
    """A workspace for tree_attention (reusable for calls of these sizes, one at a time)."""
    with _on(cache.pool):
        return _workspace(int(_serving_lib().trellis_tree_workspace_bytes(cache._ref, max(1, batch.batch), batch.max_tokens,
                                                                          q_heads)), cache.device, "tree_attention")


def tree_attention(q, cache: PagedCache, layer: int, batch: DraftBatch, workspace, scale: float = None, out=None, lse=None):
    """Attention of the drafted tokens q [n, q_heads, head_dim] over their sequences' cached prefixes and the drafts
    their masks name (written to the cache before).  scale defaults to head_dim ** -0.5.  Returns (out, lse), lse
    [n, q_heads] fp32 being the log of each softmax sum; lse=False leaves it out."""
    n, heads, dim = shape = q.shape
    index = cache.index
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=cache.device)
    if lse is None:
        lse = torch.empty((n, heads), dtype=_FP32, device=cache.device)
    qs, os_ = q.stride(), out.stride()
    inner = (dim, 1)
    if not (q.dtype is _BF16 and out.dtype is _BF16 and n == batch.n and dim == cache.head_dim and out.shape == shape and
            qs[1:] == inner and os_[1:] == inner and workspace.is_contiguous() and
            (lse is False or (lse.dtype is _FP32 and lse.shape == (n, heads) and lse.is_contiguous() and
                              lse.get_device() == index)) and
            q.get_device() == out.get_device() == workspace.get_device() == batch.index == index):
        _req_tokens(q, "q", batch.n, heads, cache.head_dim)
        _req_tokens(out, "out", n, heads, dim)
        if lse is not False:
            _req_rows(lse, "lse", _FP32, (n, heads))
            _same_device(cache.device, lse=lse)
        _req_workspace(workspace)
        _same_device(cache.device, q=q, out=out, workspace=workspace, batch=batch)
    _call("trellis_tree_attention", index, q.data_ptr(), qs[0], cache._ref, layer, batch._ref, heads,
          dim ** -0.5 if scale is None else scale, out.data_ptr(), os_[0], None if lse is False else lse.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, (None if lse is False else lse)


def new_cache_workspace(cache: PagedCache, table, pairs: int = 0) -> torch.Tensor:
    """A workspace for cache_fork (of up to `pairs` pairs) and cache_compact over the page table."""
    return _workspace(int(_serving_lib().trellis_cache_workspace_bytes(cache._ref, pairs, table.shape[1])), cache.device,
                      "cache_fork")


def cache_copy(cache: PagedCache, src, dst):
    """Copies pages src[i] to dst[i] (int32) in every layer."""
    n, index = src.shape[0], cache.index
    if not (src.dtype is _I32 and dst.dtype is _I32 and src.shape == dst.shape == (n,) and src.is_contiguous() and
            dst.is_contiguous() and src.get_device() == dst.get_device() == index):
        _req_rows(src, "src", _I32, (n,))
        _req_rows(dst, "dst", _I32, (n,))
        _same_device(cache.device, src=src, dst=dst)
    _call("trellis_cache_copy", index, cache._ref, src.data_ptr(), dst.data_ptr(), n)


def cache_fork(cache: PagedCache, table, lens, refs, parent, child, status, workspace, room: int = 0):
    """Forks, grows and frees rows of the page table in place (all int32): row child[i] becomes a copy of row
    parent[i], sharing the pages its length fills and copying the partly filled one, with room for `room` more
    positions; parent[i] = child[i] only adds the room, parent[i] = -1 frees the row.  status[i]: 0 done, 1 no room (and
    none for later pairs of the call that need fresh pages), 2 out of range."""
    rows, width = table.shape
    pairs, index = parent.shape[0], cache.index
    if not (table.dtype is _I32 and lens.dtype is _I32 and refs.dtype is _I32 and parent.dtype is _I32 and child.dtype is _I32 and
            status.dtype is _I32 and lens.shape == (rows,) and refs.shape == (cache.pages,) and
            parent.shape == child.shape == status.shape == (pairs,) and table.is_contiguous() and lens.is_contiguous() and
            refs.is_contiguous() and parent.is_contiguous() and child.is_contiguous() and status.is_contiguous() and
            workspace.is_contiguous() and table.get_device() == lens.get_device() == refs.get_device() ==
            parent.get_device() == child.get_device() == status.get_device() == workspace.get_device() == index):
        for t, name, shape in ((table, "table", (rows, width)), (lens, "lens", (rows,)), (refs, "refs", (cache.pages,)),
                               (parent, "parent", (pairs,)), (child, "child", (pairs,)), (status, "status", (pairs,))):
            _req_rows(t, name, _I32, shape)
        _req_workspace(workspace)
        _same_device(cache.device, table=table, lens=lens, refs=refs, parent=parent, child=child, status=status,
                     workspace=workspace)
    _call("trellis_cache_fork", index, cache._ref, table.data_ptr(), lens.data_ptr(), refs.data_ptr(), parent.data_ptr(),
          child.data_ptr(), status.data_ptr(), pairs, rows, width, room, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return status


def cache_compact(cache: PagedCache, table, refs, workspace, out_table=None, out_refs=None):
    """Moves the live pages (refs > 0) to the front of the pool; returns the renamed table and refs (in place unless
    out_table and out_refs are given)."""
    rows, width = table.shape
    out_table = table if out_table is None else out_table
    out_refs = refs if out_refs is None else out_refs
    index, held = cache.index, (cache.pages,)
    if not (table.dtype is _I32 and refs.dtype is _I32 and out_table.dtype is _I32 and out_refs.dtype is _I32 and
            refs.shape == held and out_table.shape == (rows, width) and out_refs.shape == held and table.is_contiguous() and
            refs.is_contiguous() and out_table.is_contiguous() and out_refs.is_contiguous() and workspace.is_contiguous() and
            table.get_device() == refs.get_device() == out_table.get_device() == out_refs.get_device() ==
            workspace.get_device() == index):
        for t, name, shape in ((table, "table", (rows, width)), (refs, "refs", held), (out_table, "out_table", (rows, width)),
                               (out_refs, "out_refs", held)):
            _req_rows(t, name, _I32, shape)
        _req_workspace(workspace)
        _same_device(cache.device, table=table, refs=refs, out_table=out_table, out_refs=out_refs, workspace=workspace)
    _call("trellis_cache_compact", index, cache._ref, table.data_ptr(), refs.data_ptr(), out_table.data_ptr(),
          out_refs.data_ptr(), rows, width, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out_table, out_refs


def cache_commit(cache: PagedCache, table, prefix, path, accepted, out_lens=None):
    """Keeps the accepted drafts of each sequence: position prefix[b] + path[b, i] moves to prefix[b] + i for
    i < accepted[b], in every layer (all int32; path [batch, max_tokens] ascending).  Returns prefix + accepted
    (out_lens may be prefix)."""
    batch, width = table.shape
    tokens = path.shape[1]
    if out_lens is None:
        out_lens = torch.empty_like(prefix)
    index, row = cache.index, (batch,)
    if not (table.dtype is _I32 and prefix.dtype is _I32 and path.dtype is _I32 and accepted.dtype is _I32 and
            out_lens.dtype is _I32 and prefix.shape == accepted.shape == out_lens.shape == row and path.shape == (batch, tokens) and
            table.is_contiguous() and prefix.is_contiguous() and path.is_contiguous() and accepted.is_contiguous() and
            out_lens.is_contiguous() and table.get_device() == prefix.get_device() == path.get_device() ==
            accepted.get_device() == out_lens.get_device() == index):
        for t, name, shape in ((table, "table", (batch, width)), (prefix, "prefix", row), (path, "path", (batch, tokens)),
                               (accepted, "accepted", row), (out_lens, "out_lens", row)):
            _req_rows(t, name, _I32, shape)
        _same_device(cache.device, table=table, prefix=prefix, path=path, accepted=accepted, out_lens=out_lens)
    _call("trellis_cache_commit", index, cache._ref, table.data_ptr(), prefix.data_ptr(), path.data_ptr(),
          accepted.data_ptr(), out_lens.data_ptr(), batch, width, tokens)
    return out_lens


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns, per row of logits."""
    logprobs: torch.Tensor      # [n, cands] fp32, of the given tokens
    lse: torch.Tensor           # [n] fp32
    entropy: torch.Tensor       # [n] fp32
    top_ids: torch.Tensor       # [n, top_k] int32, most likely first
    top_logprobs: torch.Tensor  # [n, top_k] fp32


def new_logprobs_workspace(n: int, vocab: int, top_k: int, device) -> torch.Tensor:
    """A zero-filled workspace for token_logprobs of up to n rows (reusable, one call at a time)."""
    with torch.cuda.device(device):
        return _workspace(int(_serving_lib().trellis_logprobs_workspace_bytes(n, vocab, top_k)), device, "token_logprobs")


def token_logprobs(logits, tokens, top_k: int, workspace, temperature: float = 1.0, out=None) -> TokenLogprobs:
    """Log probabilities of tokens [n, cands] int32 under softmax(logits / temperature), with each row's log of the
    softmax sum, entropy and top_k most likely tokens (equal logits: lowest index first).  logits [n, vocab] bf16 or
    fp32, rows may be apart.  out: five tensors to write, as TokenLogprobs."""
    n, vocab = logits.shape
    index, cands, stride = logits.get_device(), tokens.shape[1], logits.stride()
    dtype = logits.dtype
    if out is None:
        if index < 0:
            raise ValueError("logits must be a CUDA tensor")
        f32 = dict(dtype=_FP32, device=logits.device)
        out = (torch.empty((n, cands), **f32), torch.empty((n,), **f32), torch.empty((n,), **f32),
               torch.empty((n, top_k), dtype=_I32, device=logits.device), torch.empty((n, top_k), **f32))
    lp, ls, en, ti, tl = out
    row, given, top = (n,), (n, cands), (n, top_k)
    if not (index >= 0 and (dtype is _BF16 or dtype is _FP32) and stride[1] == 1 and tokens.dtype is _I32 and ti.dtype is _I32 and
            lp.dtype is _FP32 and ls.dtype is _FP32 and en.dtype is _FP32 and tl.dtype is _FP32 and tokens.shape == given and
            lp.shape == given and ls.shape == row and en.shape == row and ti.shape == top and tl.shape == top and
            tokens.is_contiguous() and lp.is_contiguous() and ls.is_contiguous() and en.is_contiguous() and
            ti.is_contiguous() and tl.is_contiguous() and workspace.is_contiguous() and
            tokens.get_device() == lp.get_device() == ls.get_device() == en.get_device() == ti.get_device() ==
            tl.get_device() == workspace.get_device() == index):
        if index < 0:
            raise ValueError("logits must be a CUDA tensor")
        if dtype not in (_BF16, _FP32):
            raise ValueError(f"logits has dtype {dtype}, expected torch.bfloat16 or torch.float32")
        if stride[1] != 1 and vocab > 1:
            raise ValueError("the logits of a row must be contiguous")
        for t, name, dt, shape in ((tokens, "tokens", _I32, given), (lp, "logprobs", _FP32, given), (ls, "lse", _FP32, row),
                                   (en, "entropy", _FP32, row), (ti, "top_ids", _I32, top), (tl, "top_logprobs", _FP32, top)):
            _req_rows(t, name, dt, shape)
        _req_workspace(workspace)
        _same_device(logits.device, tokens=tokens, logprobs=lp, lse=ls, entropy=en, top_ids=ti, top_logprobs=tl,
                     workspace=workspace)
    _call("trellis_token_logprobs", index, logits.data_ptr(), TRELLIS_BF16 if dtype is _BF16 else TRELLIS_F32, stride[0],
          tokens.data_ptr(), n, vocab, cands, top_k, temperature, lp.data_ptr(), ls.data_ptr(), en.data_ptr(), ti.data_ptr(),
          tl.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out if isinstance(out, TokenLogprobs) else TokenLogprobs(*out)
