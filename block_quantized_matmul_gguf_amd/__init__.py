"""GGUF quantized matmul for MI355X (gfx950): thin binding over libqmatmul.so.

y = x . W^T with W stored as GGUF Q8_0, Q4_K, Q4_0, Q5_0 or Q6_K blocks, in the two numerical
forms of the page "同一个 GGUF，CPU 和 Metal 生成的文字不一样" (section 出处):

* ``MODE_F32ACT`` (a): f32 activations, weight blocks dequantized in-kernel;
* ``MODE_QACT`` (b): activation rows quantized to Q8_0 / Q8K first, integer
  block dot products scaled by the block scales;
* ``MODE_DEQUANT``: the same page's third form (section 修法, the
  CANDLE_DEQUANTIZE_ALL switch): weights decoded to f32 once
  (``dequantize_weights``), then a plain f32 matmul (``Plan.run_dequantized``).

This module only marshals arguments: it checks dtypes, devices, contiguity and
sizes of torch tensors, then calls the C ABI (``include/qmatmul.h``) with their
device pointers and the current HIP stream.  Every step of the computation runs
in the library's HIP kernels; there is no other code path, and importing the
module fails loudly if the library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import os

Q4_0, Q5_0, Q8_0, Q4_K, Q6_K, Q8_K = 2, 6, 8, 12, 14, 15
WEIGHT_FORMATS = (Q8_0, Q4_K, Q4_0, Q5_0, Q6_K)
MODE_F32ACT, MODE_QACT, MODE_DEQUANT = 0, 1, 2
OK, EINVAL, EBLOCK, EUNSUPPORTED, ENOMEM, EHIP = 0, 1, 2, 3, 4, 5
BLOCK_VALUES = {Q8_0: 32, Q4_K: 256, Q8_K: 256, Q4_0: 32, Q5_0: 32, Q6_K: 256}
BLOCK_BYTES = {Q8_0: 34, Q4_K: 144, Q8_K: 292, Q4_0: 18, Q5_0: 22, Q6_K: 210}
ACT_FORMAT = {Q8_0: Q8_0, Q4_K: Q8_K, Q4_0: Q8_0, Q5_0: Q8_0, Q6_K: Q8_K}
GEMV_MAX_M = 8

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmatmul.so")

_p, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int

class CacheStruct(ctypes.Structure):
    """``qmm_cache`` of the header."""
    _fields_ = [("format_k", _int), ("format_v", _int), ("pages", _i64), ("page_size", _i64), ("heads", _i64), ("dim", _i64),
                ("k", _p), ("v", _p), ("batch", _i64), ("table_width", _i64), ("table", _p), ("starts", _p),
                ("lengths", _p)]


_cache_p = ctypes.POINTER(CacheStruct)

# name: (restype, argtypes) for every symbol the header declares
SIGNATURES = {
    "qmatmul_create": (_int, [ctypes.POINTER(_p), _int, _i64, _i64, _i64, _int]),
    "qmatmul_run": (_int, [_p, _p, _p, _p, _i64, _p]),
    "qmatmul_destroy": (_int, [_p]),
    "qmatmul_quantize_act": (_int, [_int, _p, _i64, _i64, _p, _p]),
    "qmatmul_quantize_weights": (_int, [_int, _p, _i64, _i64, _p, _p]),
    "qmatmul_run_block_sums": (_int, [_p, _p, _p, _p, _i64, _p]),
    "qmatmul_run_traced": (_int, [_p, _p, _p, _p, _p, _p, _i64, _p]),
    "qmatmul_dequantize_weights": (_int, [_int, _p, _i64, _i64, _p, _p]),
    "qmatmul_run_dequantized": (_int, [_p, _p, _p, _p, _i64, _p]),
    "qmatmul_run_group": (_int, [ctypes.POINTER(_p), _int, ctypes.POINTER(_p), _p, ctypes.POINTER(_p), _i64, _p]),
    "qmatmul_run_noalloc": (_int, [_int, _i64, _i64, _i64, _int, _p, _p, _p, _p]),
    "qmatmul_quantize_q4_k_search": (_int, [_p, _i64, _i64, _p, _p]),
    "qmatmul_route_experts": (_int, [_p, _int, _i64, _i64, _p, _int, _int, _int, _int, _int, _int, ctypes.c_float, _p, _p, _p]),
    "qmatmul_experts_workspace_bytes": (_i64, [_int, _int, _i64, _i64, _i64, _i64, _i64, _int]),
    "qmatmul_experts_run": (_int, [_int, _i64, _i64, _i64, _i64, _i64, _int, _int, _p, _p, _p, _p, _p, ctypes.c_size_t, _p]),
    "qmatmul_experts_glu": (_int, [_int, _i64, _i64, _i64, _i64, _i64, _int, _int, _p, _p, _p, _p, _p, _p, ctypes.c_size_t, _p]),
    "qmatmul_experts_combine": (_int, [_int, _i64, _i64, _i64, _i64, _i64, _int, _p, _p, _p, _p, _p, _p, ctypes.c_size_t, _p]),
    "qmatmul_w4_workspace_bytes": (_i64, [_i64, _i64, _i64, _i64, _int]),
    "qmatmul_w4_run": (_int, [_i64, _i64, _i64, _i64, _int, _int, _p, _p, _p, _p, _p, _p, ctypes.c_size_t, _p]),
    "qmatmul_cache_store": (_int, [_cache_p, _i64, _int, _p, _i64, _p, _i64, _p]),
    "qmatmul_cache_load": (_int, [_cache_p, _i64, _int, _p, _p, _p]),
    "qmatmul_cache_attention_workspace_bytes": (_i64, [_cache_p, _i64, _i64, _int, _int, _i64, _i64]),
    "qmatmul_cache_attention": (_int, [_cache_p, _i64, _i64, _int, _p, _i64, ctypes.c_float, _int, _i64, ctypes.c_float,
                                       _i64, _p, _p, _p, ctypes.c_size_t, _p]),
    "qmatmul_check": (_int, [_int, _i64, _i64, _i64, _int]),
    "qmatmul_row_bytes": (_i64, [_int, _i64]),
    "qmatmul_block_sums_per_row": (_i64, [_int, _i64]),
    "qmatmul_workspace_bytes": (_i64, [_int, _i64, _i64, _i64, _int]),
    "qmatmul_status_string": (ctypes.c_char_p, [_int]),
    "qmatmul_last_error": (ctypes.c_char_p, []),
    "qmatmul_version": (_int, []),
}

_lib = None


class QmmError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status} ({status_string(status)}): {message}")
        self.status = status


def lib():
    """The loaded C library (loaded once)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is not built; build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` from the repository root")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().qmatmul_status_string(status).decode()


def last_error() -> str:
    return lib().qmatmul_last_error().decode()


def _check(status: int, where: str):
    if status != OK:
        raise QmmError(status, where, last_error())


# ------------------------------------------------------------ host-only ----

def check(fmt: int, n: int, k: int, m_max: int, mode: int) -> int:
    """Validate a plan shape without touching the GPU; returns the status code."""
    return int(lib().qmatmul_check(fmt, n, k, m_max, mode))


def row_bytes(fmt: int, k: int) -> int:
    return int(lib().qmatmul_row_bytes(fmt, k))


def block_sums_per_row(fmt: int, k: int) -> int:
    return int(lib().qmatmul_block_sums_per_row(fmt, k))


def workspace_bytes(fmt: int, n: int, k: int, m_max: int, mode: int) -> int:
    return int(lib().qmatmul_workspace_bytes(fmt, n, k, m_max, mode))


# ---------------------------------------------------------- device calls ---

def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, shape, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


class Plan:
    """One weight shape and mode: ``Plan(fmt, N, K, M_max, mode)``.

    ``run(w, x)`` computes y = x . W^T.  w: uint8 tensor of N*row_bytes(fmt, K)
    bytes (any shape, contiguous), x: float32 [M, K] with M <= M_max; returns
    (or fills) float32 [M, N].  The plan's workspace is shared by its runs:
    use one plan per stream.
    """

    def __init__(self, fmt: int, n: int, k: int, m_max: int, mode: int):
        self.fmt, self.n, self.k, self.m_max, self.mode = fmt, n, k, m_max, mode
        self._h = ctypes.c_void_p()
        _check(lib().qmatmul_create(ctypes.byref(self._h), fmt, n, k, m_max, mode), "qmatmul_create")

    def _args(self, w, x):
        torch = _torch()
        _need(w, torch.uint8, None, "w")
        if w.numel() != self.n * row_bytes(self.fmt, self.k):
            raise ValueError(f"w has {w.numel()} bytes, expected {self.n * row_bytes(self.fmt, self.k)}")
        _need(x, torch.float32, None, "x")
        if x.dim() != 2 or x.shape[1] != self.k:
            raise ValueError(f"x must be [M, {self.k}], got {tuple(x.shape)}")
        return x.shape[0]

    def run(self, w, x, y=None, stream=None):
        torch = _torch()
        m = self._args(w, x)
        if y is None:
            y = torch.empty((m, self.n), dtype=torch.float32, device=x.device)
        _need(y, torch.float32, (m, self.n), "y")
        _check(lib().qmatmul_run(self._h, _ptr(w), _ptr(x), _ptr(y), m, _stream(stream)), "qmatmul_run")
        return y

    def run_dequantized(self, w_f32, x, y=None, stream=None):
        """Dequantize-all plans: y = x . W^T with W the f32 [N, K] matrix from
        ``dequantize_weights``."""
        torch = _torch()
        _need(w_f32, torch.float32, (self.n, self.k), "w_f32")
        _need(x, torch.float32, None, "x")
        if x.dim() != 2 or x.shape[1] != self.k:
            raise ValueError(f"x must be [M, {self.k}], got {tuple(x.shape)}")
        m = x.shape[0]
        if y is None:
            y = torch.empty((m, self.n), dtype=torch.float32, device=x.device)
        _need(y, torch.float32, (m, self.n), "y")
        _check(lib().qmatmul_run_dequantized(self._h, _ptr(w_f32), _ptr(x), _ptr(y), m, _stream(stream)),
               "qmatmul_run_dequantized")
        return y

    def block_sums(self, w, x, out=None, stream=None):
        torch = _torch()
        m = self._args(w, x)
        spr = block_sums_per_row(self.fmt, self.k)
        if out is None:
            out = torch.empty((m, self.n, spr), dtype=torch.int32, device=x.device)
        _need(out, torch.int32, (m, self.n, spr), "sums")
        _check(lib().qmatmul_run_block_sums(self._h, _ptr(w), _ptr(x), _ptr(out), m, _stream(stream)),
               "qmatmul_run_block_sums")
        return out

    def run_traced(self, w, x, stream=None):
        """Mode (b): the run's own kernels with their integer parts written out.
        Returns (y, sums, act): y float32 [M, N] (bit-equal to ``run``), sums
        int32 [M, N, block_sums_per_row], act uint8 [M, row_bytes of the
        activation format] (canonical Q8_0 or Q8K blocks)."""
        torch = _torch()
        m = self._args(w, x)
        spr = block_sums_per_row(self.fmt, self.k)
        y = torch.empty((m, self.n), dtype=torch.float32, device=x.device)
        sums = torch.empty((m, self.n, spr), dtype=torch.int32, device=x.device)
        act = torch.empty((m, row_bytes(ACT_FORMAT[self.fmt], self.k)), dtype=torch.uint8, device=x.device)
        _check(lib().qmatmul_run_traced(self._h, _ptr(w), _ptr(x), _ptr(y), _ptr(sums), _ptr(act), m,
                                        _stream(stream)), "qmatmul_run_traced")
        return y, sums, act

    def close(self):
        if self._h:
            _check(lib().qmatmul_destroy(self._h), "qmatmul_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            if self._h and _lib is not None:
                _lib.qmatmul_destroy(self._h)
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


GROUP_MAX = 8


def run_group(plans, ws, x, ys=None, stream=None):
    """y[i] = x . W[i]^T for plans sharing format, K and mode (one launch per
    four plans at M = 1 where the one-row kernel takes the rows); returns the
    list of outputs."""
    torch = _torch()
    if not 1 <= len(plans) <= GROUP_MAX or len(ws) != len(plans):
        raise ValueError(f"need 1..{GROUP_MAX} plans and as many weight tensors, got {len(plans)} and {len(ws)}")
    m = plans[0]._args(ws[0], x)
    for p, w in zip(plans[1:], ws[1:]):
        p._args(w, x)
    if ys is None:
        ys = [torch.empty((m, p.n), dtype=torch.float32, device=x.device) for p in plans]
    for p, y in zip(plans, ys):
        _need(y, torch.float32, (m, p.n), "y")
    n = len(plans)
    harr = (_p * n)(*[p._h for p in plans])
    warr = (_p * n)(*[_ptr(w) for w in ws])
    yarr = (_p * n)(*[_ptr(y) for y in ys])
    _check(lib().qmatmul_run_group(harr, n, warr, _ptr(x), yarr, m, _stream(stream)), "qmatmul_run_group")
    return ys


NOALLOC_SCRATCH_BYTES = 32 << 20


def run_noalloc(fmt: int, n: int, k: int, mode: int, w, x, y=None, stream=None):
    """y = x . W^T without a plan and without device allocation in the library
    (its workspace is a static device array of NOALLOC_SCRATCH_BYTES per GPU;
    calls that overlap on one GPU race).  Same arguments and values as
    ``Plan(fmt, n, k, M, mode).run(w, x)``; allocates ``y`` here only when it is
    not given."""
    torch = _torch()
    _need(w, torch.uint8, None, "w")
    rb = row_bytes(fmt, k)
    if rb < 0 or w.numel() != n * rb:
        raise ValueError(f"w has {w.numel()} bytes, expected {n} rows of {rb}")
    _need(x, torch.float32, None, "x")
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"x must be [M, {k}], got {tuple(x.shape)}")
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _need(y, torch.float32, (m, n), "y")
    _check(lib().qmatmul_run_noalloc(fmt, n, k, m, mode, _ptr(w), _ptr(x), _ptr(y), _stream(stream)),
           "qmatmul_run_noalloc")
    return y


def quantize_act(act_fmt: int, x, out=None, stream=None):
    """Canonical Q8_0 (34 B / 32) or Q8K (292 B / 256) blocks of the rows of x
    (float32 [M, K] on the GPU); returns uint8 [M, row_bytes]."""
    torch = _torch()
    _need(x, torch.float32, None, "x")
    m, k = x.shape
    rb = row_bytes(act_fmt, k)
    if rb < 0:
        raise ValueError(f"K={k} is not a multiple of the block size of format {act_fmt}")
    if out is None:
        out = torch.empty((m, rb), dtype=torch.uint8, device=x.device)
    _need(out, torch.uint8, (m, rb), "out")
    _check(lib().qmatmul_quantize_act(act_fmt, _ptr(x), m, k, _ptr(out), _stream(stream)), "qmatmul_quantize_act")
    return out


def quantize_weights(fmt: int, w, out=None, stream=None):
    """GGUF blocks of the rows of w (float32 [N, K] on the GPU); returns uint8 [N, row_bytes]."""
    torch = _torch()
    _need(w, torch.float32, None, "w")
    n, k = w.shape
    rb = row_bytes(fmt, k)
    if rb < 0:
        raise ValueError(f"K={k} is not a multiple of the block size of format {fmt}")
    if out is None:
        out = torch.empty((n, rb), dtype=torch.uint8, device=w.device)
    _need(out, torch.uint8, (n, rb), "out")
    _check(lib().qmatmul_quantize_weights(fmt, _ptr(w), n, k, _ptr(out), _stream(stream)), "qmatmul_quantize_weights")
    return out


def quantize_q4_k_search(w, out=None, stream=None):
    """Q4_K blocks of the rows of w (float32 [N, K] on the GPU) with the
    least-squares search for each sub-block's scale and min."""
    torch = _torch()
    _need(w, torch.float32, None, "w")
    n, k = w.shape
    rb = row_bytes(Q4_K, k)
    if rb < 0:
        raise ValueError(f"K={k} is not a multiple of 256")
    if out is None:
        out = torch.empty((n, rb), dtype=torch.uint8, device=w.device)
    _need(out, torch.uint8, (n, rb), "out")
    _check(lib().qmatmul_quantize_q4_k_search(_ptr(w), n, k, _ptr(out), _stream(stream)), "qmatmul_quantize_q4_k_search")
    return out


def dequantize_weights(fmt: int, w, n: int, k: int, out=None, stream=None):
    """f32 [N, K] of GGUF weight blocks w (uint8, N*row_bytes(fmt, K) bytes, on
    the GPU): the exact dequantized values rounded once to f32."""
    torch = _torch()
    _need(w, torch.uint8, None, "w")
    rb = row_bytes(fmt, k)
    if rb < 0:
        raise ValueError(f"K={k} is not a multiple of the block size of format {fmt}")
    if w.numel() != n * rb:
        raise ValueError(f"w has {w.numel()} bytes, expected {n * rb}")
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _need(out, torch.float32, (n, k), "out")
    _check(lib().qmatmul_dequantize_weights(fmt, _ptr(w), n, k, _ptr(out), _stream(stream)),
           "qmatmul_dequantize_weights")
    return out


# ------------------------------------- mixture of experts, 4-bit groups ----
#
# These calls take no plan.  A call's scratch tensor and, unless the caller
# gives them, its outputs come from torch's allocator on the stream of the
# call (``stream``, a torch.cuda.Stream, or the current one), so calls may
# overlap on different streams and be captured in graphs that run side by side.
# As with torch's own work on a second stream, the caller has that stream wait
# for inputs made on another, and keeps them until it is done with them.
# An output that the caller gives must not overlap an input (QmmError).

F32, F16, BF16 = 0, 1, 2
SCORES = {"softmax": 0, "sigmoid": 1}
ACTS = {"silu": 0, "gelu": 1}
EXPERTS_RUN, EXPERTS_GLU, EXPERTS_COMBINE, EXPERTS_RUN_SLOTS = 0, 1, 2, 3
_TYPES = None


def _type_of(t, name):
    global _TYPES
    if _TYPES is None:
        torch = _torch()
        _TYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _tensor(t, dtype, dims, name, device=None):
    """Checks a tensor argument: on the GPU (on ``device``), contiguous, of
    ``dtype`` (None: a float type) and ``dims`` dimensions."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dims is not None and t.dim() not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, shape, dtype, device, name):
    """A given output, checked, or a new one on the current stream."""
    if t is None:
        return _torch().empty(shape, dtype=dtype, device=device)
    _tensor(t, dtype, None, name, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _current_stream(torch, index):
    """The handle of device ``index``'s current stream (torch's own shortcut to
    it: building a Stream object would cost a fifth of a small call)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _on_device(device, stream, body):
    """Runs body(stream handle) with ``device`` current and ``stream`` (None:
    that device's current stream) as the stream of allocations."""
    torch = _torch()
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return body(_current_stream(torch, device.index))
        with torch.cuda.device(device):
            return body(_current_stream(torch, device.index))
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


@functools.lru_cache(maxsize=4096)
def _experts_workspace(product, fmt, e, n, k, t, top_k, code):
    return int(lib().qmatmul_experts_workspace_bytes(product, fmt, e, n, k, t, top_k, code))


@functools.lru_cache(maxsize=4096)
def _w4_workspace(n, k, m, group, code):
    return int(lib().qmatmul_w4_workspace_bytes(n, k, m, group, code))


def _scratch(nbytes, device):
    """(pointer, bytes, the tensor that owns them) of a call's workspace; none
    for sizes that the call itself will refuse."""
    if nbytes <= 0:
        return None, 0, None
    ws = _torch().empty(nbytes, dtype=_torch().uint8, device=device)
    return ws.data_ptr(), nbytes, ws


def route_experts(logits, top_k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int | None = None,
                  group_top: int = 1, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """The experts of each row of logits (float32, float16 or bfloat16 [T, E]):
    (ids int32 [T, top_k], weights float32 [T, top_k]).

    Scores are softmax or sigmoid of the logits; the choice is by score + bias
    (float32 [E]), within the ``top_groups`` best of ``groups`` groups of
    neighbouring experts (a group's score: the sum of its ``group_top`` best
    choices), ties to the lower index.  Experts with a -inf or NaN logit or bias
    are never chosen; slots left over have id -1 and weight 0.  Weights are the
    scores, divided by their sum if ``renormalize``, times ``scale``; a bias
    does not change the scores, softmax's sum included."""
    torch = _torch()
    _tensor(logits, None, (2,), "logits")
    code = _type_of(logits, "logits")
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    dev = logits.device
    t, e = logits.shape
    if bias is not None:
        _tensor(bias, torch.float32, (1,), "bias", dev)
        if bias.shape[0] != e:
            raise ValueError(f"bias must have shape ({e},), got {tuple(bias.shape)}")

    def body(s):
        i = _out(ids, (t, top_k), torch.int32, dev, "ids")
        w = _out(weights, (t, top_k), torch.float32, dev, "weights")
        _check(lib().qmatmul_route_experts(
            logits.data_ptr(), code, t, e, None if bias is None else bias.data_ptr(), SCORES[score], top_k, groups,
            groups if top_groups is None else top_groups, group_top, int(renormalize), scale, i.data_ptr(),
            w.data_ptr(), s), "qmatmul_route_experts")
        return i, w

    if not 1 <= top_k <= min(64, e):
        raise ValueError(f"top_k must be in 1..{min(64, e)}, got {top_k}")
    return _on_device(dev, stream, body)


def _expert_args(fmt, w, x, ids, x_dims, name):
    """Checks what the experts' products share; (E, N, K, T, top_k, type)."""
    torch = _torch()
    _tensor(x, None, x_dims, name)
    code = _type_of(x, name)
    dev = x.device
    _tensor(ids, torch.int32, (2,), "ids", dev)
    t, k = ids.shape
    if x.shape[0] != t or (x.dim() == 3 and x.shape[1] != k):
        raise ValueError(f"{name} {tuple(x.shape)} and ids {tuple(ids.shape)} differ in tokens or slots")
    kk = x.shape[-1]
    rb = row_bytes(fmt, kk)
    if rb < 0:
        raise ValueError(f"K={kk} is not a multiple of the block size of format {fmt}")
    e = n = None
    for t_w, w_name in w:
        _tensor(t_w, torch.uint8, (3,), w_name, dev)
        if t_w.shape[2] != rb or (e is not None and (t_w.shape[0] != e or t_w.shape[1] != n)):
            raise ValueError(f"{w_name} must be [E, N, {rb}] uint8, got {tuple(t_w.shape)}")
        e, n = t_w.shape[0], t_w.shape[1]
    return e, n, kk, t, k, code


def experts_matmul(fmt: int, w, x, ids, y=None, stream=None):
    """y[t, s] = x[t] . W[ids[t, s]]^T: the products of tokens with the weights
    of their experts.  w: uint8 [E, N, row_bytes(fmt, K)] GGUF blocks; x:
    float32, float16 or bfloat16 [T, K], or [T, top_k, K] with a row per slot;
    ids: int32 [T, top_k], values outside 0..E-1 meaning no expert (zeros).
    Returns [T, top_k, N] in x's type."""
    e, n, kk, t, k, code = _expert_args(fmt, ((w, "w"),), x, ids, (2, 3), "x")
    dev = x.device

    def body(s):
        out = _out(y, (t, k, n), x.dtype, dev, "y")
        ws, nb, keep = _scratch(_experts_workspace(EXPERTS_RUN if x.dim() == 2 else EXPERTS_RUN_SLOTS, fmt, e, n, kk, t, k,
                                                   code), dev)
        _check(lib().qmatmul_experts_run(fmt, e, n, kk, t, k, code, int(x.dim() == 3), w.data_ptr(), x.data_ptr(),
                                         ids.data_ptr(), out.data_ptr(), ws, nb, s), "qmatmul_experts_run")
        return out

    return _on_device(dev, stream, body)


def experts_glu(fmt: int, w_gate, w_up, x, ids, act: str = "silu", h=None, stream=None):
    """h[t, s] = act(x[t] . Wg^T) * (x[t] . Wu^T) with the gate and up weights
    of expert ids[t, s] (both uint8 [E, N, row_bytes(fmt, K)]); act "silu" or
    "gelu" (the tanh form).  Returns [T, top_k, N] in x's type."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    e, n, kk, t, k, code = _expert_args(fmt, ((w_gate, "w_gate"), (w_up, "w_up")), x, ids, (2,), "x")
    dev = x.device

    def body(s):
        out = _out(h, (t, k, n), x.dtype, dev, "h")
        ws, nb, keep = _scratch(_experts_workspace(EXPERTS_GLU, fmt, e, n, kk, t, k, code), dev)
        _check(lib().qmatmul_experts_glu(fmt, e, n, kk, t, k, code, ACTS[act], w_gate.data_ptr(), w_up.data_ptr(),
                                         x.data_ptr(), ids.data_ptr(), out.data_ptr(), ws, nb, s), "qmatmul_experts_glu")
        return out

    return _on_device(dev, stream, body)


def experts_combine(fmt: int, w, h, ids, weights, y=None, stream=None):
    """y[t] = sum_s weights[t, s] * (h[t, s] . W[ids[t, s]]^T): the experts'
    last product and the weighted sum over a token's slots.  h: [T, top_k, K],
    weights: float32 [T, top_k].  Returns [T, N] in h's type."""
    e, n, kk, t, k, code = _expert_args(fmt, ((w, "w"),), h, ids, (3,), "h")
    dev = h.device
    _tensor(weights, _torch().float32, (2,), "weights", dev)
    if tuple(weights.shape) != (t, k):
        raise ValueError(f"weights must have shape {(t, k)}, got {tuple(weights.shape)}")

    def body(s):
        out = _out(y, (t, n), h.dtype, dev, "y")
        ws, nb, keep = _scratch(_experts_workspace(EXPERTS_COMBINE, fmt, e, n, kk, t, k, code), dev)
        _check(lib().qmatmul_experts_combine(fmt, e, n, kk, t, k, code, w.data_ptr(), h.data_ptr(), ids.data_ptr(),
                                             weights.data_ptr(), out.data_ptr(), ws, nb, s), "qmatmul_experts_combine")
        return out

    return _on_device(dev, stream, body)


def w4_matmul(q, scales, x, zeros=None, y=None, stream=None):
    """y = x . W^T with 4-bit weights in groups: W[n, k] = scales[n, k // G] *
    (q[n, k] - z), z = zeros[n, k // G] or 8.  q: uint8 [N, K/2], element 2i in
    the low nibble of byte i; scales: float32, float16 or bfloat16 [N, K/G],
    G a multiple of 32; zeros: uint8 [N, K/G]; x: float32, float16 or bfloat16
    [M, K].  Returns [M, N] in x's type."""
    torch = _torch()
    _tensor(x, None, (2,), "x")
    code = _type_of(x, "x")
    dev = x.device
    m, kk = x.shape
    _tensor(q, torch.uint8, (2,), "q", dev)
    n = q.shape[0]
    if q.shape[1] * 2 != kk:
        raise ValueError(f"q must be [N, {kk // 2}] for K={kk}, got {tuple(q.shape)}")
    _tensor(scales, None, (2,), "scales", dev)
    scode = _type_of(scales, "scales")
    ng = scales.shape[1]
    if scales.shape[0] != n or ng == 0 or kk % ng:
        raise ValueError(f"scales must be [{n}, K / group], got {tuple(scales.shape)} for K={kk}")
    if zeros is not None:
        _tensor(zeros, torch.uint8, (2,), "zeros", dev)
        if zeros.shape != scales.shape:
            raise ValueError(f"zeros must have the scales' shape {tuple(scales.shape)}, got {tuple(zeros.shape)}")
    g = kk // ng

    def body(s):
        out = _out(y, (m, n), x.dtype, dev, "y")
        ws, nb, keep = _scratch(_w4_workspace(n, kk, m, g, code), dev)
        _check(lib().qmatmul_w4_run(n, kk, m, g, code, scode, q.data_ptr(), scales.data_ptr(),
                                    None if zeros is None else zeros.data_ptr(), x.data_ptr(), out.data_ptr(), ws, nb, s),
               "qmatmul_w4_run")
        return out

    return _on_device(dev, stream, body)


# ------------------------------------------- quantized cache, attention ----
#
# Streams, scratch and outputs as with the experts' calls above.

def _cache_args(fmt_k, fmt_v, k_cache, v_cache, table, starts, lengths):
    """Checks a cache and a batch; their ``qmm_cache``."""
    torch = _torch()
    u8, i32 = torch.uint8, torch.int32
    try:  # what good arguments need, in few steps; the others are told what is wrong below
        index = k_cache.get_device()
        good = (index >= 0 and k_cache.dtype is u8 and k_cache.dim() == 4 and k_cache.is_contiguous()
                and v_cache.get_device() == index and v_cache.dtype is u8 and v_cache.is_contiguous()
                and table.get_device() == index and table.dtype is i32 and table.dim() == 2 and table.is_contiguous()
                and starts.get_device() == index and starts.dtype is i32 and starts.dim() == 1 and starts.is_contiguous()
                and lengths.get_device() == index and lengths.dtype is i32 and lengths.dim() == 1 and lengths.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        _tensor(k_cache, u8, (4,), "k_cache")
        for t, dtype, dims, name in ((v_cache, u8, 4, "v_cache"), (table, i32, 2, "table"), (starts, i32, 1, "starts"),
                                     (lengths, i32, 1, "lengths")):
            _tensor(t, dtype, (dims,), name, k_cache.device)
    if (fmt_k != Q8_0 and fmt_k != Q4_0) or (fmt_v != Q8_0 and fmt_v != Q4_0):
        raise ValueError(f"cache formats are Q8_0 and Q4_0, got {fmt_k} and {fmt_v}")
    pages, heads, page_size, rk = k_cache.shape
    blocks, rest = divmod(rk, BLOCK_BYTES[fmt_k])
    if rk == 0 or rest:
        raise ValueError(f"k_cache must be [pages, heads, page size, row bytes], got {tuple(k_cache.shape)}")
    want = (pages, heads, page_size, blocks * BLOCK_BYTES[fmt_v])
    if v_cache.shape != want:
        raise ValueError(f"v_cache must have shape {want}, got {tuple(v_cache.shape)}")
    batch, width = table.shape
    if starts.shape[0] != batch + 1 or lengths.shape[0] != batch:
        raise ValueError(f"for {batch} sequences starts must be [{batch + 1}] and lengths [{batch}], got "
                         f"{tuple(starts.shape)} and {tuple(lengths.shape)}")
    return CacheStruct(fmt_k, fmt_v, pages, page_size, heads, 32 * blocks, k_cache.data_ptr(), v_cache.data_ptr(), batch, width,
                       table.data_ptr(), starts.data_ptr(), lengths.data_ptr())


@functools.lru_cache(maxsize=4096)
def _attention_workspace(fmt_k, fmt_v, pages, page_size, heads, dim, batch, width, t, q_heads, code, causal, window, max_length):
    c = CacheStruct(fmt_k, fmt_v, pages, page_size, heads, dim, None, None, batch, width, None, None, None)
    return int(lib().qmatmul_cache_attention_workspace_bytes(c, t, q_heads, code, causal, window, max_length))


def _token_rows(t, heads, dim, name, device):
    """Checks a tensor of tokens [T, heads (None: any), dim], contiguous but for
    the step from token to token; (T, heads, that step, type)."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's GPU, {device}, got {t.device}")
    code = _type_of(t, name)
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {dim}], got {tuple(t.shape)}")
    n, h, _ = t.shape
    step, across, along = t.stride()
    if n == 0:
        return n, h, h * dim, code
    if along != 1 or (h > 1 and across != dim):
        raise ValueError(f"{name} must be contiguous within a token, got strides {t.stride()}")
    return n, h, h * dim if n == 1 else step, code


def cache_store(fmt_k: int, fmt_v: int, k_cache, v_cache, k, v, table, starts, lengths, stream=None):
    """Quantizes the tokens' keys and values k, v (float32, float16 or bfloat16
    [T, heads, dim], of one type; the step from token to token is free) into the
    pages of their sequences, in place.

    k_cache, v_cache: uint8 [pages, heads, page_size, row_bytes(fmt, dim)], fmt
    Q8_0 or Q4_0, page_size a multiple of 64, dim 64, 96, 128 or 256 (the bytes
    of 64 tokens are in the library's own order: ``cache_load`` reads them).
    table int32 [B, W]: the pages of each sequence; starts int32 [B + 1]: where
    its rows of k and v begin; lengths int32 [B]: its tokens in the cache, these
    rows included as the last ones.  Rows of no sequence and positions without a
    page are left out."""
    c = _cache_args(fmt_k, fmt_v, k_cache, v_cache, table, starts, lengths)
    dev = k_cache.device
    t, _, k_step, code = _token_rows(k, c.heads, c.dim, "k", dev)
    tv, _, v_step, code_v = _token_rows(v, c.heads, c.dim, "v", dev)
    if tv != t or code_v != code:
        raise ValueError(f"k and v must have one shape and type, got {tuple(k.shape)} {k.dtype} and {tuple(v.shape)} {v.dtype}")

    def body(s):
        _check(lib().qmatmul_cache_store(c, t, code, k.data_ptr(), k_step, v.data_ptr(), v_step, s), "qmatmul_cache_store")

    _on_device(dev, stream, body)


def cache_load(fmt_k: int, fmt_v: int, k_cache, v_cache, table, starts, lengths, tokens: int, dtype=None, k=None, v=None,
               stream=None):
    """The keys and values of the batch's rows read back: (k, v), each [tokens,
    heads, dim] of ``dtype`` (float32 unless given).  Cache, table, starts and
    lengths as in ``cache_store``; tokens: rows of the outputs (starts[B]; rows
    of no sequence are not written).  With starts the running sum of lengths
    these are the whole sequences.  Positions without a page give zeros."""
    torch = _torch()
    c = _cache_args(fmt_k, fmt_v, k_cache, v_cache, table, starts, lengths)
    dev = k_cache.device
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    dtype = dtype or (torch.float32 if k is None else k.dtype)
    shape = (tokens, c.heads, c.dim)

    def body(s):
        ko = _out(k, shape, dtype, dev, "k")
        vo = torch.empty_like(ko) if v is None else _out(v, shape, dtype, dev, "v")
        _check(lib().qmatmul_cache_load(c, tokens, _type_of(ko, "k"), ko.data_ptr(), vo.data_ptr(), s), "qmatmul_cache_load")
        return ko, vo

    return _on_device(dev, stream, body)


def cache_attention(fmt_k: int, fmt_v: int, k_cache, v_cache, q, table, starts, lengths, scale: float | None = None,
                    causal: bool = True, window: int = 0, softcap: float = 0.0, max_length: int = 0, out=None, lse=None,
                    stream=None):
    """Attention of the batch's rows over the cache: out[n, h] = sum_j p_j v_j
    with p the softmax of scale * q[n, h] . k_j over the positions that the row
    sees (causal: up to its own; window: its last ``window``), capped first as
    softcap * tanh(x / softcap) if softcap > 0.

    q: float32, float16 or bfloat16 [T, q_heads, dim] (the step from token to
    token is free), q_heads a multiple of the cache's heads; scale: 1 /
    sqrt(dim) unless given.  Cache, table, starts and lengths as in
    ``cache_store``: one new token per sequence, many, or both side by side.
    max_length: a bound on lengths if known (0: what the table can hold), by which
    the work is split (results are right under any, but one far above the lengths
    costs time: 4096 positions 13 us, with a table of 131072 and no bound 25 us).
    Returns [T, q_heads, dim] in q's type; rows that see
    nothing are zeros, rows of no sequence are not written.  lse: float32 [T,
    q_heads] to be filled with ln sum exp(score)."""
    torch = _torch()
    c = _cache_args(fmt_k, fmt_v, k_cache, v_cache, table, starts, lengths)
    dev = k_cache.device
    dim = c.dim
    t, heads, step, code = _token_rows(q, None, dim, "q", dev)
    if lse is not None:
        _out(lse, (t, heads), torch.float32, dev, "lse")
    if scale is None:
        scale = dim ** -0.5
    pages, cache_heads, page_size, _ = k_cache.shape
    batch, width = table.shape
    causal = 1 if causal else 0

    def body(s):
        o = torch.empty_like(q) if out is None and q.is_contiguous() else _out(out, (t, heads, dim), q.dtype, dev, "out")
        ws, nb, keep = _scratch(_attention_workspace(fmt_k, fmt_v, pages, page_size, cache_heads, dim, batch, width, t, heads,
                                                     code, causal, window, max_length), dev)
        _check(lib().qmatmul_cache_attention(c, t, heads, code, q.data_ptr(), step, scale, causal, window, softcap,
                                             max_length, o.data_ptr(), None if lse is None else lse.data_ptr(), ws, nb, s),
               "qmatmul_cache_attention")
        return o

    return _on_device(dev, stream, body)
