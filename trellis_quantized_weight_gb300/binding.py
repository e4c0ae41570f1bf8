"""Thin ctypes binding of libtrellis_gb300.so (the C ABI in include/trellis.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their data pointers and the current CUDA stream are handed to the
library, and a non-zero status raises ``TrellisError``.  Every step of the
decode and product runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

from . import build as _build

_lock = threading.Lock()
_lib = None

STATUS = {
    0: "TRELLIS_OK", -1: "TRELLIS_ERR_NULL", -2: "TRELLIS_ERR_SHAPE", -3: "TRELLIS_ERR_UNSUPPORTED",
    -4: "TRELLIS_ERR_ALIGN", -5: "TRELLIS_ERR_CUDA", -6: "TRELLIS_ERR_TIMEOUT", -7: "TRELLIS_ERR_WORKSPACE",
}

# Exported functions: name -> (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_LL = ctypes.c_longlong
_D = ctypes.c_double
SIGNATURES = {
    "trellis_abi_version": (_I, []),
    "trellis_status_string": (ctypes.c_char_p, [_I]),
    "trellis_decode": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "trellis_gemm": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "trellis_gemm_workspace_size": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "trellis_gemm_ws": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "trellis_gemm_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "trellis_device_status": (_I, [_P]),
    "trellis_selftest_wait_timeout": (_I, [_P]),
    "trellis_gemm_gateup": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "trellis_gemm_gateup_workspace_size": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "trellis_gemm_packed": (_I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "trellis_gemm_packed_workspace_size": (_I, [_P, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "trellis_rope_table": (_I, [_P, _I, _I, _D, _D, _D, _D, _D, _D, _P]),
    "trellis_kv_append": (_I, [_P, _LL, _P, _LL, _P, _LL, _P, _P, _P, *[_I] * 9, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "trellis_kv_attention": (_I, [_P, _LL, _P, _P, _P, *[_I] * 9, ctypes.c_float, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "trellis_kv_attention_workspace_size": (_I, [*[_I] * 6, ctypes.POINTER(_SZ)]),
    "trellis_lora_add": (_I, [*[_P] * 7, *[_I] * 6, _P, _P, _SZ, _P]),
    "trellis_lora_add_workspace_size": (_I, [*[_I] * 6, ctypes.POINTER(_SZ)]),
}


class TrellisError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def library_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: the CUDA library has not been built "
                    "(run trellis_quantized_weight_gb300.build.build())")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
        return _lib


def status_string(status: int) -> str:
    try:
        return load().trellis_status_string(status).decode()
    except Exception:  # the message is only decoration
        return STATUS.get(status, "TRELLIS_ERR_UNKNOWN")


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise TrellisError(rc, where)


# ---- raw ABI calls (integer pointers; used by tests and the benchmark) ----
def abi_decode(codes_ptr, scales_ptr, K, N, k, L, T, out_ptr, stream) -> int:
    return load().trellis_decode(codes_ptr, scales_ptr, K, N, k, L, T, out_ptr, stream)


def abi_gemm(x_ptr, codes_ptr, scales_ptr, M, K, N, k, L, T, out_ptr, stream) -> int:
    return load().trellis_gemm(x_ptr, codes_ptr, scales_ptr, M, K, N, k, L, T, out_ptr, stream)


def abi_gemm_ws(x_ptr, codes_ptr, scales_ptr, M, K, N, k, L, T, out_ptr, ws_ptr, ws_bytes, stream) -> int:
    return load().trellis_gemm_ws(x_ptr, codes_ptr, scales_ptr, M, K, N, k, L, T, out_ptr, ws_ptr,
                                  ws_bytes, stream)


def gemm_workspace_bytes(M, K, N, k, L=12, T=256) -> int:
    n = ctypes.c_size_t(0)
    _check(load().trellis_gemm_workspace_size(M, K, N, k, L, T, ctypes.byref(n)),
           "trellis_gemm_workspace_size")
    return int(n.value)


def gemm_gateup_workspace_bytes(M, K, N, k, L=12, T=256) -> int:
    n = ctypes.c_size_t(0)
    _check(load().trellis_gemm_gateup_workspace_size(M, K, N, k, L, T, ctypes.byref(n)),
           "trellis_gemm_gateup_workspace_size")
    return int(n.value)


def gemm_packed_workspace_bytes(rows, K, N, k, L=12, T=256) -> int:
    r = (ctypes.c_int * len(rows))(*rows)
    n = ctypes.c_size_t(0)
    _check(load().trellis_gemm_packed_workspace_size(r, len(rows), K, N, k, L, T, ctypes.byref(n)),
           "trellis_gemm_packed_workspace_size")
    return int(n.value)


# ---- torch-facing API ------------------------------------------------------
def _torch():
    import torch
    return torch


def _require(t, name, dtypes, ndim):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


class _Workspace:
    """The zero-filled workspace of a device and stream, reused across calls and grown as needed.

    It is allocated and zero-filled on the stream the calls run on, so stream order alone makes the
    fill land first and lets torch's caching allocator recycle an outgrown buffer once the calls
    enqueued before it are done: no host synchronisation.  One buffer per stream also keeps calls on
    different streams off each other's counters and partial sums.  Calls of several host threads on
    one stream take turns: a call may enqueue two kernels that hand data on in the workspace, and
    the buffer must not be replaced between the look at it and the launch.

    A captured call's replays use the buffer that it was captured with, so one that is in a graph is
    kept for good when it is outgrown.  A call that needs a new buffer while it is captured takes one
    of the graph's own memory, zero-filled by every replay, which no other call gets."""
    __slots__ = ("lock", "buf", "ptr", "size", "in_graph", "kept")

    def __init__(self):
        self.lock = threading.Lock()
        self.buf, self.ptr, self.size = None, None, 0
        self.in_graph, self.kept = False, []

    def grow(self, nbytes, index, stream, capturing):
        """A buffer of at least nbytes; the caller holds it until its launch."""
        buf = _zeros(max(nbytes, 256), index, stream)
        if not capturing:
            if self.in_graph:
                self.kept.append(self.buf)
            self.buf, self.ptr, self.size, self.in_graph = buf, buf.data_ptr(), buf.numel(), False
        return buf


_ws_cache: dict = {}


def _zeros(nbytes, index, stream):
    torch = _torch()
    with torch.cuda.stream(stream):             # None: the current stream
        return torch.zeros(nbytes, dtype=torch.uint8, device=f"cuda:{index}")


def _current_device():
    return (_types or _torch_types())[8]()


def _on_device(index):
    return _torch().cuda.device(index)


def _enqueue(fn, args, index, stream):
    """fn(*args, stream) on the tensors' device, as _launch: the library launches on the thread's current device."""
    if _current_device() != index:
        with _on_device(index):
            return _enqueue(fn, args, index, stream)
    _check(fn(*args, _raw_stream(index, stream)), fn.__name__)


def _is_capturing(stream):
    is_capturing = (_types or _torch_types())[7]
    if stream is None:
        return is_capturing()
    with _torch().cuda.stream(stream):
        return is_capturing()


def _launch(fn, args, index, stream, need, ask=True):
    """fn(*args, workspace, its bytes, stream) with the stream's workspace.  need() is the size of it; with ask=False
    it is not looked up unless the call refuses the workspace at hand."""
    if _current_device() != index:
        with _on_device(index):
            return _launch(fn, args, index, stream, need, ask)
    handle = _raw_stream(index, stream)
    ws = _ws_cache.get((index, handle)) or _ws_cache.setdefault((index, handle), _Workspace())
    least = max(need(), 256) if ask else 0
    with ws.lock:
        capturing = _is_capturing(stream)
        rc = -7
        if ws.size >= least:
            if capturing and ws.buf is not None:
                ws.in_graph = True
            rc = fn(*args, ws.ptr, ws.size, handle)
        if rc == -7:
            buf = ws.grow(least or need(), index, stream, capturing)
            rc = fn(*args, buf.data_ptr(), buf.numel(), handle)
    _check(rc, fn.__name__)


def _empty(shape, dtype, index, stream):
    """A result for a call on `stream` (None: the current one).  Memory that the current stream may still be using
    is not given to a call on another, and what it gets is not handed on before the current stream is done with it."""
    torch = _torch()
    device = f"cuda:{index}"
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(index))
    return out


def _used_on(stream, *tensors):
    """What the tensors hold is not given to others before the work that `stream` has by then is done."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def decode(codes, scales, K: int, k: int, L: int = 12, T: int = 256, out=None, stream=None):
    """Dense bf16 weights [N, K] from packed codes [N, K*k/32] and bf16 scales [N]."""
    torch = _torch()
    _require(codes, "codes", (torch.int32, torch.uint32), 2)
    _require(scales, "scales", (torch.bfloat16,), 1)
    N = codes.shape[0]
    if codes.shape[1] * 32 != K * k or scales.numel() != N:
        raise ValueError("codes must be [N, K*k/32] and scales [N]")
    if out is None:
        out = _empty((N, K), torch.bfloat16, codes.get_device(), stream)
    _require(out, "out", (torch.bfloat16,), 2)
    if tuple(out.shape) != (N, K):
        raise ValueError("out must be [N, K]")
    _enqueue(load().trellis_decode, (codes.data_ptr(), scales.data_ptr(), K, N, k, L, T, out.data_ptr()), codes.get_device(),
             stream)
    _used_on(stream, codes, scales, out)
    return out


def gemm(x, codes, scales, k: int, L: int = 12, T: int = 256, out=None, stream=None):
    """out [M, N] bf16 = x [M, K] times the decoded weights [N, K] transposed."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,), 2)
    _require(codes, "codes", (torch.int32, torch.uint32), 2)
    _require(scales, "scales", (torch.bfloat16,), 1)
    M, K = x.shape
    N = codes.shape[0]
    if codes.shape[1] * 32 != K * k or scales.numel() != N:
        raise ValueError("codes must be [N, K*k/32] and scales [N]")
    if out is None:
        out = _empty((M, N), torch.bfloat16, x.get_device(), stream)
    _require(out, "out", (torch.bfloat16,), 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    _launch(load().trellis_gemm_ws, (x.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, K, N, k, L, T, out.data_ptr()),
            x.get_device(), stream, lambda: gemm_workspace_bytes(M, K, N, k, L, T))
    _used_on(stream, x, codes, scales, out)
    return out


def gemm_gateup(x, codes_gate, scales_gate, codes_up, scales_up, k: int, act: bool = True, L: int = 12,
                T: int = 256, stream=None):
    """The two projections that share x: returns (gate [M, N], up [M, N], act [M, N] or None)
    with act = bf16(silu(gate) * up)."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,), 2)
    for name, c, sc in (("gate", codes_gate, scales_gate), ("up", codes_up, scales_up)):
        _require(c, f"codes_{name}", (torch.int32, torch.uint32), 2)
        _require(sc, f"scales_{name}", (torch.bfloat16,), 1)
    M, K = x.shape
    N = codes_gate.shape[0]
    if tuple(codes_up.shape) != tuple(codes_gate.shape) or codes_gate.shape[1] * 32 != K * k:
        raise ValueError("codes_gate and codes_up must both be [N, K*k/32]")
    if scales_gate.numel() != N or scales_up.numel() != N:
        raise ValueError("scales must be [N]")
    g, u, a = (_empty((M, N), torch.bfloat16, x.get_device(), stream) if wanted else None for wanted in (True, True, act))
    _launch(load().trellis_gemm_gateup, (x.data_ptr(), codes_gate.data_ptr(), scales_gate.data_ptr(), codes_up.data_ptr(),
                                         scales_up.data_ptr(), M, K, N, k, L, T, g.data_ptr(), u.data_ptr(),
                                         a.data_ptr() if act else None),
            x.get_device(), stream, lambda: gemm_gateup_workspace_bytes(M, K, N, k, L, T))
    _used_on(stream, x, codes_gate, scales_gate, codes_up, scales_up, g, u, a)
    return g, u, a


def gemm_packed(xs, codes, scales, k: int, L: int = 12, T: int = 256, outs=None, stream=None):
    """Token packing: one product for several groups of activation rows sharing the
    weights.  xs: list of bf16 [rows_g, K]; returns the list of bf16 [rows_g, N]."""
    torch = _torch()
    xs = list(xs)
    if not xs:
        raise ValueError("xs must hold at least one group")
    for i, x in enumerate(xs):
        _require(x, f"xs[{i}]", (torch.bfloat16,), 2)
    _require(codes, "codes", (torch.int32, torch.uint32), 2)
    _require(scales, "scales", (torch.bfloat16,), 1)
    K = xs[0].shape[1]
    N = codes.shape[0]
    if any(x.shape[1] != K for x in xs) or codes.shape[1] * 32 != K * k or scales.numel() != N:
        raise ValueError("every x must be [rows, K] with codes [N, K*k/32] and scales [N]")
    rows = [int(x.shape[0]) for x in xs]
    if outs is None:
        outs = [_empty((r, N), torch.bfloat16, xs[0].get_device(), stream) for r in rows]
    for i, (o, r) in enumerate(zip(outs, rows)):
        _require(o, f"outs[{i}]", (torch.bfloat16,), 2)
        if tuple(o.shape) != (r, N):
            raise ValueError(f"outs[{i}] must be [{r}, {N}]")
    xp = (ctypes.c_void_p * len(xs))(*[x.data_ptr() for x in xs])
    op = (ctypes.c_void_p * len(outs))(*[o.data_ptr() for o in outs])
    rp = (ctypes.c_int * len(rows))(*rows)
    _launch(load().trellis_gemm_packed, (xp, rp, len(rows), codes.data_ptr(), scales.data_ptr(), K, N, k, L, T, op),
            xs[0].get_device(), stream, lambda: gemm_packed_workspace_bytes(rows, K, N, k, L, T))
    _used_on(stream, *xs, codes, scales, *outs)
    return outs


# ---- the attention block's cache and adapters --------------------------------
class KVCache(NamedTuple):
    """A paged key/value cache: e4m3 codes [pages, kv_heads, page_size, head_dim] and, for each
    16 tokens of a page and head, a power-of-two scale, float32 [pages, kv_heads, page_size / 16].
    The functions below take any such four tensors in this order."""
    k: object
    v: object
    k_scale: object
    v_scale: object


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """An empty cache of `pages` pages."""
    torch = _torch()
    codes = [torch.zeros((pages, kv_heads, page_size, head_dim), dtype=torch.uint8, device=device)
             .view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((pages, kv_heads, page_size // 16), dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*codes, *scales)


def rope_table(positions: int, rot: int, base: float = 10000.0, stretch: float = 1.0, original: int = 0,
               low: float = 1.0, high: float = 32.0, gain: float = 1.0, device="cuda", stream=None):
    """cos and sin of the rotary positions, float32 [positions, rot], for kv_append.  stretch > 1 slows
    the pairs for longer contexts: all of them, or with `original` > 0 only those that make few
    turns over that many positions (fully at `low` turns, not at all from `high` on)."""
    torch = _torch()
    if not isinstance(positions, int) or positions < 1 or not isinstance(rot, int) or rot < 1:
        raise ValueError("positions and rot must be positive ints")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    index = torch.cuda.current_device() if device.index is None else device.index
    table = _empty((positions, rot), torch.float32, index, stream)
    _enqueue(load().trellis_rope_table, (table.data_ptr(), positions, rot, base, stretch, float(original), low, high, gain),
             index, stream)
    _used_on(stream, table)
    return table


# The calls below are made several times a layer and step, so their host side is kept
# short: one query of the stream, no query of the workspace's size unless the one at hand
# is refused.
def _raw_stream(index, stream):
    if stream is not None:
        return stream.cuda_stream
    return (_types or _torch_types())[6](index)


_types = None


def _torch_types():
    """Tensor, bfloat16, float32, int32, float8_e4m3fn, empty, the current stream's handle, whether it is capturing,
    and the current device."""
    global _types
    if _types is None:
        torch = _torch()
        _types = (torch.Tensor, torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.empty,
                  torch._C._cuda_getCurrentRawStream, torch._C._cuda_isCurrentStreamCapturing, torch._C._cuda_getDevice)
    return _types


def _require_rows(t, name, index):
    types = _types or _torch_types()
    if not isinstance(t, types[0]) or t.get_device() != index:
        raise ValueError(f"{name} must be a tensor on cuda:{index}")
    shape = t.shape
    if t.dtype != types[1] or len(shape) != 3:
        raise ValueError(f"{name} must be a bfloat16 [tokens, heads, head_dim] tensor")
    row, head, one = t.stride()
    if (one != 1 or (shape[1] > 1 and head != shape[2])) and t.numel():
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    # the stride of a single row is arbitrary: the row's own length then
    return shape, row if shape[0] > 1 else shape[1] * shape[2]


def _require_on(t, name, dtype, ndim, index):
    if not isinstance(t, _types[0]) or index < 0 or t.get_device() != index or t.dtype != dtype \
            or not t.is_contiguous() or len(shape := t.shape) != ndim:
        raise ValueError(f"{name} must be a contiguous {ndim}-d {dtype} tensor on one CUDA device")
    return shape


def _require_cache(cache, starts, kv_len, pages):
    """Checks a cache and its sequences' arrays; returns (codes' shape, sequences, table columns, device index)."""
    Tensor, _, f32, i32, f8 = (_types or _torch_types())[:5]
    k, v, ks, vs = cache
    if not isinstance(k, Tensor) or (index := k.get_device()) < 0:
        raise ValueError("the cache must be CUDA tensors")
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or k.dtype != f8 or v.dtype != f8:
        raise ValueError("cache codes must be float8_e4m3fn [pages, kv_heads, page_size, head_dim]")
    want = (shape[0], shape[1], shape[2] // 16)
    if ks.shape != want or vs.shape != want or ks.dtype != f32 or vs.dtype != f32:
        raise ValueError("cache scales must be float32 [pages, kv_heads, page_size / 16]")
    if v.get_device() != index or ks.get_device() != index or vs.get_device() != index:
        raise ValueError("the cache must be on one device")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache must be contiguous")
    n, = _require_on(starts, "starts", i32, 1, index)
    seqs, = _require_on(kv_len, "kv_len", i32, 1, index)
    rows, cols = _require_on(pages, "pages", i32, 2, index)
    if n != seqs + 1 or rows != seqs:
        raise ValueError("starts must be [S + 1], kv_len [S] and pages [S, columns]")
    return shape, seqs, cols, index


def _output(out, name, shape, index, device, stream):
    types = _types or _torch_types()
    if out is None:
        return types[5](shape, dtype=types[1], device=device) if stream is None else _empty(shape, types[1], index, stream)
    if not isinstance(out, types[0]) or out.shape != shape or out.dtype != types[1] or out.get_device() != index \
            or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 {tuple(shape)} tensor on cuda:{index}")
    return out


def kv_append(cache, k, v, starts, kv_len, pages, q=None, rope=None, interleaved: bool = False, max_q=None, q_out=None,
              stream=None):
    """Put a step's keys and values into the paged cache, rotated on the way, and return its rotated
    queries (None without q).

    k, v: bf16 [tokens, kv_heads, head_dim]; q: bf16 [tokens, q_heads, head_dim] (rows may be
    strided, as slices of one projection's output are).  starts int32 [S + 1]: the rows of each
    sequence; kv_len int32 [S]: its tokens with these; pages int32 [S, columns]: its pages.
    rope: float32 [positions, rot] from rope_table, or None; positions past it are rotated as its last.
    max_q: rows of the sequence that has most, all by default; it shapes the launch, results do not depend on it.
    The cache is updated in place."""
    (num_pages, hk, page, d), seqs, cols, index = _require_cache(cache, starts, kv_len, pages)
    k_shape, k_stride = _require_rows(k, "k", index)
    v_shape, v_stride = _require_rows(v, "v", index)
    tokens = k_shape[0]
    if k_shape != (tokens, hk, d) or v_shape != k_shape:
        raise ValueError(f"k and v must be [tokens, {hk}, {d}]")
    hq, q_ptr, q_stride, out_ptr = hk, None, 0, None
    if q is not None:
        q_shape, q_stride = _require_rows(q, "q", index)
        hq = q_shape[1]
        if q_shape[0] != tokens or q_shape[2] != d:
            raise ValueError(f"q must be [{tokens}, heads, {d}]")
        q_out = _output(q_out, "q_out", q_shape, index, k.device, stream)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope_ptr, rows, rot = None, 0, 0
    if rope is not None:
        rows, rot = _require_on(rope, "rope", _types[2], 2, index)
        rope_ptr = rope.data_ptr()
    if seqs == 0 or tokens == 0:
        return q_out
    _enqueue((_lib or load()).trellis_kv_append,
             (q_ptr, q_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, starts.data_ptr(), kv_len.data_ptr(),
              pages.data_ptr(), tokens, seqs, tokens if max_q is None else max_q, cols, num_pages, hq, hk, d, page, rope_ptr,
              rows, rot, 1 if interleaved else 0, cache[0].data_ptr(), cache[1].data_ptr(), cache[2].data_ptr(),
              cache[3].data_ptr(), out_ptr), index, stream)
    if stream is not None:
        _used_on(stream, *cache, k, v, q, starts, kv_len, pages, rope, q_out)
    return q_out


def kv_attention_workspace_bytes(tokens, seqs, max_q, q_heads, kv_heads, head_dim) -> int:
    n = ctypes.c_size_t(0)
    _check(load().trellis_kv_attention_workspace_size(tokens, seqs, max_q, q_heads, kv_heads, head_dim,
                                                      ctypes.byref(n)), "trellis_kv_attention_workspace_size")
    return int(n.value)


def kv_attention(q, cache, starts, kv_len, pages, scale=None, window: int = 0, max_q=None, out=None, stream=None):
    """Causal attention of a step's queries over the paged cache: bf16 [tokens, q_heads, head_dim].

    q: bf16 [tokens, q_heads, head_dim], rows may be strided; the rest as kv_append, whose
    tokens the cache holds by now.  scale: of the scores, 1 / sqrt(head_dim) by default;
    window: how many tokens a row sees, itself included (0: all before it).  max_q, the rows of the
    sequence that has most, chooses the kernel of the whole call: give it for single tokens and
    drafts (64 single tokens take 172 us with it, 389 without), and where prompt chunks stand
    beside many single tokens make a call for each."""
    (num_pages, hk, page, d), seqs, cols, index = _require_cache(cache, starts, kv_len, pages)
    shape, q_stride = _require_rows(q, "q", index)
    tokens, hq = shape[0], shape[1]
    if shape[2] != d:
        raise ValueError(f"q must be [tokens, heads, {d}]")
    dev = q.device
    out = _output(out, "out", shape, index, dev, stream)
    if seqs == 0 or tokens == 0:
        return out
    most = tokens if max_q is None else max_q
    _launch((_lib or load()).trellis_kv_attention,
            (q.data_ptr(), q_stride, starts.data_ptr(), kv_len.data_ptr(), pages.data_ptr(), tokens, seqs, most, cols,
             num_pages, hq, hk, d, page, d ** -0.5 if scale is None else scale, window, cache[0].data_ptr(),
             cache[1].data_ptr(), cache[2].data_ptr(), cache[3].data_ptr(), out.data_ptr()),
            index, stream, lambda: kv_attention_workspace_bytes(tokens, seqs, most, hq, hk, d), ask=False)
    if stream is not None:
        _used_on(stream, q, *cache, starts, kv_len, pages, out)
    return out


def lora_add_workspace_bytes(M, K, N, R, adapters, segments) -> int:
    n = ctypes.c_size_t(0)
    _check(load().trellis_lora_add_workspace_size(M, K, N, R, adapters, segments, ctypes.byref(n)),
           "trellis_lora_add_workspace_size")
    return int(n.value)


def lora_add(y, x, a, b, scales, starts, which, out=None, stream=None):
    """y + scales[w] * (x A[w]^T) B[w]^T for each request's adapter w: bf16 [M, N].

    y: bf16 [M, N], the output of the projection that the requests share; x: bf16 [M, K], its
    input; a: bf16 [adapters, R, K]; b: bf16 [adapters, N, R]; scales: float32 [adapters].
    starts int32 [S + 1]: the rows of each request; which int32 [S]: its adapter, -1 for none.
    out may be y."""
    Tensor, bf16, f32, i32 = (_types or _torch_types())[:4]
    if not isinstance(y, Tensor):
        raise ValueError("y must be a CUDA tensor")
    dev, index = y.device, y.get_device()
    shape = _require_on(y, "y", bf16, 2, index)
    x_rows, K = _require_on(x, "x", bf16, 2, index)
    n_ad, R, k_a = _require_on(a, "a", bf16, 3, index)
    b_shape = _require_on(b, "b", bf16, 3, index)
    n_scales, = _require_on(scales, "scales", f32, 1, index)
    n, = _require_on(starts, "starts", i32, 1, index)
    segments, = _require_on(which, "which", i32, 1, index)
    M, N = shape
    if x_rows != M or k_a != K or b_shape != (n_ad, N, R) or n_scales != n_ad:
        raise ValueError("y must be [M, N], x [M, K], a [adapters, R, K], b [adapters, N, R] and scales [adapters]")
    if n != segments + 1:
        raise ValueError("starts must be [S + 1] with which [S]")
    out = _output(out, "out", shape, index, dev, stream)
    if M == 0:
        return out
    _launch((_lib or load()).trellis_lora_add,
            (y.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(), scales.data_ptr(), starts.data_ptr(),
             which.data_ptr(), M, K, N, R, n_ad, segments, out.data_ptr()),
            index, stream, lambda: lora_add_workspace_bytes(M, K, N, R, n_ad, segments), ask=False)
    if stream is not None:
        _used_on(stream, y, x, a, b, scales, starts, which, out)
    return out
