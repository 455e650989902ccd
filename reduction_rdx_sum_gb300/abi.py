"""Python binding of librdx.so: the C-ABI entry points under the same names.

Argument marshalling only: each function checks the tensors it is given,
passes their device pointers, sizes and the current CUDA stream to the C
entry point, and raises ``RdxError`` on a non-zero status.  All arithmetic
happens in the CUDA kernels.  If the library has not been built (see
``reduction_rdx_sum_gb300.build``), every call raises; there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

import torch

from .build import LIB

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "rdx.h")

RDX_OK = 0
RDX_ERR_INVALID_ARG = 1
RDX_ERR_CUDA = 2
RDX_ERR_ALLOC = 3
RDX_ERR_UNSUPPORTED_DEVICE = 4

_lock = threading.Lock()
_lib = None


class RdxError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})" + (f": {detail}" if detail else ""))
        self.status = status


def declared_symbols() -> list[str]:
    """Names of the functions include/rdx.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(rdx_[a-z0-9_]+)\s*\(", text)))


def load(path: str | None = None) -> ctypes.CDLL:
    """Open librdx.so (once) and declare the C signatures.  RDX_LIBRARY may
    name another build of it (the checked build, for instance)."""
    global _lib
    path = path or os.environ.get("RDX_LIBRARY") or LIB
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is not built; run reduction_rdx_sum_gb300.build.build() "
                               "(or __graft_entry__.build()) first")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        for name in ("rdx_sum_f32", "rdx_sumsq_f32", "rdx_sum_bf16_f32acc", "rdx_sumsq_bf16_f32acc",
                     "rdx_sum_i32_i64", "rdx_sum_sumsq_f32", "rdx_sum_sumsq_bf16_f32acc", "rdx_max_f32",
                     "rdx_max_i32", "rdx_sum_f32_noalloc"):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [vp, i64, vp, vp], i32
        lib.rdx_rowsum_f32.argtypes, lib.rdx_rowsum_f32.restype = [vp, i64, i64, vp, vp], i32
        lib.rdx_rowsum_strided_f32.argtypes = [vp, i64, i64, i64, vp, vp]
        lib.rdx_rowsum_strided_f32.restype = i32
        lib.rdx_workspace_bytes.argtypes, lib.rdx_workspace_bytes.restype = [], ctypes.c_size_t
        lib.rdx_reduce_kernels.argtypes, lib.rdx_reduce_kernels.restype = [i32, i64], i32
        lib.rdx_rowsum_kernels.argtypes, lib.rdx_rowsum_kernels.restype = [i64, i64], i32
        lib.rdx_reduce_ws.argtypes = [i32, vp, i64, vp, vp, ctypes.c_size_t, vp]
        lib.rdx_reduce_ws.restype = i32
        lib.rdx_bank_probe.argtypes, lib.rdx_bank_probe.restype = [i32, i32, vp, vp, vp], i32
        lib.rdx_bank_probe_loads_per_iter.argtypes, lib.rdx_bank_probe_loads_per_iter.restype = [], i32
        lib.rdx_debug_build.argtypes, lib.rdx_debug_build.restype = [], i32
        lib.rdx_debug_violations.argtypes, lib.rdx_debug_violations.restype = [vp, i32], i32
        lib.rdx_wait_timeouts.argtypes, lib.rdx_wait_timeouts.restype = [vp, i32], i32
        lib.rdx_debug_stage_timeout.argtypes, lib.rdx_debug_stage_timeout.restype = [vp, i64, i64, vp, vp], i32
        lib.rdx_ladder_partials_f32.argtypes = [i32, vp, i64, vp, vp]
        lib.rdx_ladder_partials_f32.restype = i32
        lib.rdx_ladder_num_partials.argtypes, lib.rdx_ladder_num_partials.restype = [i32, i64], i64
        lib.rdx_ladder_sum_f32.argtypes, lib.rdx_ladder_sum_f32.restype = [i32, vp, i64, vp, vp, vp], i32
        lib.rdx_shard_range.argtypes = [i64, i32, i32, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        lib.rdx_shard_range.restype = i32
        lib.rdx_combine_max_parts.argtypes, lib.rdx_combine_max_parts.restype = [], i32
        for name in ("rdx_combine_f32", "rdx_combine_f32x2", "rdx_combine_i64"):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [vp, i32, vp, vp], i32
        for name in ("rdx_qk_norm_rope", "rdx_qk_norm_rope_grad", "rdx_kv_write", "rdx_kv_read", "rdx_kv_attend"):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [vp, vp], i32
        lib.rdx_qk_norm_rope_grad_workspace_bytes.argtypes = [i32]
        lib.rdx_qk_norm_rope_grad_workspace_bytes.restype = ctypes.c_size_t
        lib.rdx_kv_attend_workspace_bytes.argtypes = [vp]
        lib.rdx_kv_attend_workspace_bytes.restype = ctypes.c_size_t
        lib.rdx_status_string.argtypes, lib.rdx_status_string.restype = [i32], ctypes.c_char_p
        lib.rdx_last_cuda_error.argtypes, lib.rdx_last_cuda_error.restype = [], ctypes.c_char_p
        lib.rdx_shutdown.argtypes, lib.rdx_shutdown.restype = [], None
        lib.rdx_release_stream.argtypes, lib.rdx_release_stream.restype = [vp], i32
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().rdx_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != RDX_OK:
        raise RdxError(fn, status, load().rdx_last_cuda_error().decode())


try:  # the current stream's cudaStream_t by device index, without building a Stream object
    _current_raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # pragma: no cover - builds without the accessor
    def _current_raw_stream(index: int) -> int:
        return int(torch.cuda.current_stream(index).cuda_stream)


def _launch(fn, device, stream, *args) -> int:
    """fn(*args, stream handle) with `device` current: the C entry points
    launch on the current device, in `stream` (default: the current stream
    of `device`).  The device is switched only when it is not current."""
    index = device.index if isinstance(device, torch.device) else int(device)
    if index == torch.cuda.current_device():
        return fn(*args, _current_raw_stream(index) if stream is None else int(stream.cuda_stream))
    with torch.cuda.device(index):
        return fn(*args, _current_raw_stream(index) if stream is None else int(stream.cuda_stream))


def _input(x: torch.Tensor, dtypes, what: str) -> torch.Tensor:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{what}: expected dtype in {dtypes}, got {x.dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return x


def _output(out, like: torch.Tensor, dtype, shape) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if not out.is_cuda or out.dtype != dtype or tuple(out.shape) != tuple(shape) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")
    return out


def _scalar(name: str, x: torch.Tensor, dtypes, out_dtype, out, stream, shape=()) -> torch.Tensor:
    lib = load()
    x = _input(x, dtypes, name)
    out = _output(out, x, out_dtype, shape)
    st = _launch(getattr(lib, name), x.device, stream, x.data_ptr(), x.numel(), out.data_ptr())
    _check(name, st)
    return out


_BF16 = (torch.bfloat16, torch.int16, torch.uint16) if hasattr(torch, "uint16") else (torch.bfloat16, torch.int16)


def rdx_sum_f32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the sum of a float32 tensor."""
    return _scalar("rdx_sum_f32", x, (torch.float32,), torch.float32, out, stream)


def rdx_sumsq_f32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the sum of squares of a float32 tensor."""
    return _scalar("rdx_sumsq_f32", x, (torch.float32,), torch.float32, out, stream)


def rdx_sum_bf16_f32acc(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the sum of a bfloat16 tensor (or its raw 16-bit patterns)."""
    return _scalar("rdx_sum_bf16_f32acc", x, _BF16, torch.float32, out, stream)


def rdx_sumsq_bf16_f32acc(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the sum of squares of a bfloat16 tensor."""
    return _scalar("rdx_sumsq_bf16_f32acc", x, _BF16, torch.float32, out, stream)


def rdx_sum_i32_i64(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d int64 tensor: the exact sum of an int32 tensor."""
    return _scalar("rdx_sum_i32_i64", x, (torch.int32,), torch.int64, out, stream)


def rdx_sum_sumsq_f32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(2,) float32 tensor [sum, sum of squares] of a float32 tensor, one pass."""
    return _scalar("rdx_sum_sumsq_f32", x, (torch.float32,), torch.float32, out, stream, shape=(2,))


def rdx_sum_sumsq_bf16_f32acc(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(2,) float32 tensor [sum, sum of squares] of a bfloat16 tensor, one pass."""
    return _scalar("rdx_sum_sumsq_bf16_f32acc", x, _BF16, torch.float32, out, stream, shape=(2,))


def rdx_max_f32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the maximum of a float32 tensor (NaNs skipped; empty gives -Inf)."""
    return _scalar("rdx_max_f32", x, (torch.float32,), torch.float32, out, stream)


def rdx_max_i32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d int32 tensor: the maximum of an int32 tensor (empty gives -2^31)."""
    return _scalar("rdx_max_i32", x, (torch.int32,), torch.int32, out, stream)


def rdx_rowsum_f32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(rows,) float32 tensor: per-row sums of a contiguous 2-D float32 tensor."""
    lib = load()
    x = _input(x, (torch.float32,), "rdx_rowsum_f32")
    if x.dim() != 2:
        raise ValueError("rdx_rowsum_f32: expected a 2-D tensor")
    rows, cols = x.shape
    out = _output(out, x, torch.float32, (rows,))
    st = _launch(lib.rdx_rowsum_f32, x.device, stream, x.data_ptr(), rows, cols, out.data_ptr())
    _check("rdx_rowsum_f32", st)
    return out


def rdx_rowsum_strided_f32(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(rows,) float32 tensor: per-row sums of a 2-D float32 tensor whose rows
    are contiguous (stride(1) == 1) and start every stride(0) elements, such
    as a column slice of a wider matrix."""
    lib = load()
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float32 or x.dim() != 2:
        raise TypeError("rdx_rowsum_strided_f32: expected a 2-D float32 CUDA tensor")
    rows, cols = x.shape
    if cols > 1 and x.stride(1) != 1:
        raise ValueError("rdx_rowsum_strided_f32: rows must be contiguous (stride(1) == 1)")
    ld = x.stride(0) if rows > 1 else cols
    out = _output(out, x, torch.float32, (rows,))
    st = _launch(lib.rdx_rowsum_strided_f32, x.device, stream, x.data_ptr(), rows, cols, ld, out.data_ptr())
    _check("rdx_rowsum_strided_f32", st)
    return out


# RDX_OP_* codes of include/rdx.h, by operation name.
OP_CODES = {"sum_f32": 0, "sumsq_f32": 1, "sum_bf16": 2, "sumsq_bf16": 3, "sum_i32": 4,
            "sum_sumsq_f32": 5, "sum_sumsq_bf16": 6, "max_f32": 7, "max_i32": 8}
_OP_IN = {0: (torch.float32,), 1: (torch.float32,), 2: _BF16, 3: _BF16, 4: (torch.int32,), 5: (torch.float32,),
          6: _BF16, 7: (torch.float32,), 8: (torch.int32,)}
_OP_OUT = {0: (torch.float32, ()), 1: (torch.float32, ()), 2: (torch.float32, ()), 3: (torch.float32, ()),
           4: (torch.int64, ()), 5: (torch.float32, (2,)), 6: (torch.float32, (2,)), 7: (torch.float32, ()),
           8: (torch.int32, ())}


def rdx_workspace_bytes() -> int:
    return int(load().rdx_workspace_bytes())


def rdx_reduce_kernels(op, n: int) -> int:
    """Kernels one call of scalar reduction ``op`` (name or RDX_OP_* code) on n elements enqueues."""
    return int(load().rdx_reduce_kernels(OP_CODES[op] if isinstance(op, str) else int(op), n))


def rdx_rowsum_kernels(rows: int, cols: int) -> int:
    """Kernels one rdx_rowsum_f32 call on a rows x cols matrix enqueues."""
    return int(load().rdx_rowsum_kernels(rows, cols))


def rdx_reduce_ws(op, x: torch.Tensor, workspace: torch.Tensor, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Scalar reduction ``op`` (a name of OP_CODES or an RDX_OP_* code) with a
    caller-owned workspace (a CUDA tensor of at least rdx_workspace_bytes()
    bytes, zero-filled before its first use)."""
    lib = load()
    code = OP_CODES[op] if isinstance(op, str) else int(op)
    if code not in _OP_IN:
        raise ValueError(f"rdx_reduce_ws: unknown op {op}")
    x = _input(x, _OP_IN[code], "rdx_reduce_ws")
    dt, shape = _OP_OUT[code]
    out = _output(out, x, dt, shape)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("rdx_reduce_ws: workspace must be a contiguous CUDA tensor")
    st = _launch(lib.rdx_reduce_ws, x.device, stream, code, x.data_ptr(), x.numel(), out.data_ptr(),
                 workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check("rdx_reduce_ws", st)
    return out


def rdx_bank_probe(pattern: int, iters: int = 256, device=None, stream=None) -> float:
    """Clock cycles per shared-memory load instruction of the page's bank
    pattern ``pattern`` (0..9), measured by one warp on the GPU."""
    lib = load()
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    cycles = torch.zeros(1, dtype=torch.int64, device=device)
    sink = torch.zeros(32, dtype=torch.int32, device=device)
    st = _launch(lib.rdx_bank_probe, device, stream, pattern, iters, cycles.data_ptr(), sink.data_ptr())
    _check("rdx_bank_probe", st)
    return cycles.item() / (iters * lib.rdx_bank_probe_loads_per_iter())


def rdx_ladder_num_partials(version: int, n: int) -> int:
    return int(load().rdx_ladder_num_partials(version, n))


def rdx_ladder_partials_f32(version: int, x: torch.Tensor, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Per-block partials of the page's block-reduction ``version`` (1..5)."""
    lib = load()
    x = _input(x, (torch.float32,), "rdx_ladder_partials_f32")
    nb = lib.rdx_ladder_num_partials(version, x.numel())
    if nb < 0:
        raise ValueError(f"rdx_ladder_partials_f32: bad version {version}")
    out = _output(out, x, torch.float32, (nb,))
    st = _launch(lib.rdx_ladder_partials_f32, x.device, stream, version, x.data_ptr(), x.numel(), out.data_ptr())
    _check("rdx_ladder_partials_f32", st)
    return out


def rdx_sum_f32_noalloc(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the sum of a float32 tensor, computed with the
    library's static scratch instead of an allocated workspace (for callers
    that may not allocate device memory; calls must not overlap on the GPU)."""
    return _scalar("rdx_sum_f32_noalloc", x, (torch.float32,), torch.float32, out, stream)


def rdx_ladder_sum_f32(version: int, x: torch.Tensor, out: torch.Tensor | None = None,
                       partials: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the sum of a float32 tensor by the page's block
    reduction ``version`` (1..5), its per-block partials (left in
    ``partials``) added on the device in the same launch."""
    lib = load()
    x = _input(x, (torch.float32,), "rdx_ladder_sum_f32")
    nb = lib.rdx_ladder_num_partials(version, x.numel())
    if nb < 0:
        raise ValueError(f"rdx_ladder_sum_f32: bad version {version}")
    partials = _output(partials, x, torch.float32, (nb,))
    out = _output(out, x, torch.float32, ())
    st = _launch(lib.rdx_ladder_sum_f32, x.device, stream, version, x.data_ptr(), x.numel(), partials.data_ptr(),
                 out.data_ptr())
    _check("rdx_ladder_sum_f32", st)
    return out


def rdx_shard_range(n: int, parts: int, rank: int, granule: int) -> tuple[int, int]:
    """(lo, hi): the chunk of rank ``rank`` among ``parts`` sharing ``n``
    elements cut in whole granules of ``granule`` elements (host only)."""
    lo, hi = ctypes.c_int64(0), ctypes.c_int64(0)
    _check("rdx_shard_range", load().rdx_shard_range(n, parts, rank, granule, ctypes.byref(lo), ctypes.byref(hi)))
    return int(lo.value), int(hi.value)


def rdx_combine_max_parts() -> int:
    return int(load().rdx_combine_max_parts())


def _combine(name: str, parts: torch.Tensor, dtype, width: int, out, stream) -> torch.Tensor:
    lib = load()
    parts = _input(parts, (dtype,), name)
    if parts.numel() % width:
        raise ValueError(f"{name}: expected {width} values per partial")
    p = parts.numel() // width
    out = _output(out, parts, dtype, () if width == 1 else (width,))
    st = _launch(getattr(lib, name), parts.device, stream, parts.data_ptr(), p, out.data_ptr())
    _check(name, st)
    return out


def rdx_combine_f32(parts: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d float32 tensor: the float32 partials ``parts`` added in index (rank) order."""
    return _combine("rdx_combine_f32", parts, torch.float32, 1, out, stream)


def rdx_combine_f32x2(parts: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(2,) float32 tensor: the [sum, sum of squares] pairs ``parts`` (p x 2)
    added component-wise in rank order."""
    return _combine("rdx_combine_f32x2", parts, torch.float32, 2, out, stream)


def rdx_combine_i64(parts: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """0-d int64 tensor: the int64 partials ``parts`` added (modulo 2^64)."""
    return _combine("rdx_combine_i64", parts, torch.int64, 1, out, stream)


def rdx_shutdown() -> None:
    load().rdx_shutdown()


def rdx_release_stream(stream=None, device=None) -> bool:
    """Free the library's workspace for ``stream`` (default: the current
    stream) on ``device`` (default: the current device); True if one was
    freed.  Call after the stream's work has completed."""
    index = torch.cuda.current_device() if device is None else torch.device(device).index
    with torch.cuda.device(index):
        handle = _current_raw_stream(index) if stream is None else int(stream.cuda_stream)
        return bool(load().rdx_release_stream(handle))


def rdx_debug_build() -> bool:
    """True when the loaded library is the checked build (RDX_DEBUG=1)."""
    return bool(load().rdx_debug_build())


def rdx_debug_violations(reset: bool = False) -> int:
    """Out-of-range accesses the checked build caught (0 in a normal build)."""
    count = ctypes.c_uint64(0)
    _check("rdx_debug_violations", load().rdx_debug_violations(ctypes.byref(count), int(reset)))
    return int(count.value)


def rdx_wait_timeouts(reset: bool = False) -> int:
    """Staging waits of the narrow-row kernel that gave up on the current
    device since the last reset (synchronizes the device)."""
    count = ctypes.c_uint64(0)
    _check("rdx_wait_timeouts", load().rdx_wait_timeouts(ctypes.byref(count), int(reset)))
    return int(count.value)


def rdx_debug_stage_timeout(x: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Test hook: one narrow-row tile of the 2-D float32 tensor x (rows *
    cols <= 6144) whose staging wait cannot complete, so that it gives up
    after one second; out (rows float32 values) is left unwritten."""
    if x.dim() != 2 or x.dtype != torch.float32 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous 2-D float32 CUDA tensor")
    rows, cols = x.shape
    _check("rdx_debug_stage_timeout",
           _launch(load().rdx_debug_stage_timeout, x.device, stream, x.data_ptr(), rows, cols, out.data_ptr()))


# Entry points by operation name, for the tests and the bench.
SCALAR_OPS = {
    "sum_f32": rdx_sum_f32,
    "sumsq_f32": rdx_sumsq_f32,
    "sum_bf16": rdx_sum_bf16_f32acc,
    "sumsq_bf16": rdx_sumsq_bf16_f32acc,
    "sum_i32": rdx_sum_i32_i64,
    "max_f32": rdx_max_f32,
    "max_i32": rdx_max_i32,
}

# One-pass [sum, sum of squares] entry points by input type.
PAIR_OPS = {
    "f32": rdx_sum_sumsq_f32,
    "bf16": rdx_sum_sumsq_bf16_f32acc,
}


# ---- heads: norms with rotation, the 8-bit cache, attention over it ---------------------------------------------------
#
# Rows are heads: [tokens, heads, head_dim] tensors whose last dimension is contiguous and whose other strides are free.
# These calls marshal their tensors in the extension module _marshal (csrc/marshal.cpp), which checks them, allocates
# results on the call's stream and passes the C argument structs to the library opened by load().

TYPE_CODES = {torch.float32: 0, torch.bfloat16: 1}
KV_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}

_KV_ATTEND_ARGS = struct.Struct("@PPPPqiiii" + "Pqq" * 2 + "PPPPQ" + "qqqq" + "iif0q")

MARSHALLED = ("rdx_qk_norm_rope", "rdx_qk_norm_rope_grad", "rdx_qk_norm_rope_grad_workspace_bytes", "rdx_kv_write",
              "rdx_kv_read", "rdx_kv_attend", "rdx_kv_attend_workspace_bytes")  # in bind's order

_module = None


def _marshal():
    """The marshalling module, bound to the library (once)."""
    global _module
    if _module is None:
        lib = load()
        try:
            from . import _marshal as module
        except ImportError as e:
            raise RuntimeError("the marshalling module is not built; run reduction_rdx_sum_gb300.build.build() "
                               f"(or __graft_entry__.build()) first ({e})") from e
        built_for = getattr(module, "torch_version", "another version")
        if built_for != torch.__version__:
            raise RuntimeError(f"the marshalling module was built for PyTorch {built_for}, this is "
                               f"{torch.__version__}; run reduction_rdx_sum_gb300.build.build() again")
        address = [ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in MARSHALLED]
        module.bind(*address, KVCache, _check)
        _module = module
    return _module


def rdx_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                     positions: torch.Tensor | None, cos: torch.Tensor | None, sin: torch.Tensor | None,
                     eps: float = 1e-6, interleaved: bool = False, q_out: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(q_out, k_out): the heads of q [tokens, q_heads, head_dim] and k [tokens, k_heads, head_dim] (float32 or
    bfloat16) divided by their root mean square, times the float32 weights, and turned by the angles of row
    positions[t] of the float32 tables cos and sin [positions, rot_dim / 2] (None: no rotation).  q_out and k_out may
    be q and k.  Where q, k or a weight requires a gradient, autograd gets it from rdx_qk_norm_rope_grad; a q_out or
    k_out of the caller's is refused then, and tables that require one always are."""
    y = (_module or _marshal()).qk_norm_rope(q, k, q_weight, k_weight, positions, cos, sin, eps, interleaved, q_out,
                                             k_out, stream)
    return y if y is not NotImplemented else _followed_norm_rope(q, k, q_weight, k_weight, positions, cos, sin, eps,
                                                                 interleaved, q_out, k_out, stream)


def _followed_norm_rope(q, k, q_weight, k_weight, positions, cos, sin, eps, interleaved, q_out, k_out, stream):
    """rdx_qk_norm_rope where a tensor requires a gradient."""
    if any(x is not None and x.requires_grad for x in (cos, sin)):
        raise RuntimeError("rdx_qk_norm_rope: there is no gradient of the tables cos and sin; pass them detached")
    if q_out is not None or k_out is not None:
        raise RuntimeError("rdx_qk_norm_rope: a q_out or k_out of the caller's would lose the gradients that q, k, the "
                           "weights or the outputs require; pass none, or call it under torch.no_grad()")
    with torch.cuda.stream(stream):  # None: as it is
        return _NormRope.apply(q, k, q_weight, k_weight, positions, cos, sin, eps, interleaved)


class _NormRope(torch.autograd.Function):
    """rdx_qk_norm_rope for autograd."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, cos, sin, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, cos, sin)
        ctx.eps, ctx.interleaved = eps, interleaved
        return _marshal().qk_norm_rope(q, k, q_weight, k_weight, positions, cos, sin, eps, interleaved, None, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        # a loss's gradient may be one value for all: the rows' last dimension is contiguous here
        dq_out, dk_out = (d if d.stride(2) == 1 else d.contiguous() for d in (dq_out, dk_out))
        return (*rdx_qk_norm_rope_grad(dq_out, dk_out, *ctx.saved_tensors, eps=ctx.eps, interleaved=ctx.interleaved),
                None, None, None, None, None)


def rdx_qk_norm_rope_grad_workspace_bytes(head_dim: int) -> int:
    return int(load().rdx_qk_norm_rope_grad_workspace_bytes(head_dim))


def rdx_qk_norm_rope_grad(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          q_weight: torch.Tensor, k_weight: torch.Tensor, positions: torch.Tensor | None,
                          cos: torch.Tensor | None, sin: torch.Tensor | None, eps: float = 1e-6,
                          interleaved: bool = False, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                          dq_weight: torch.Tensor | None = None, dk_weight: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, ...]:
    """(dq, dk, dq_weight, dk_weight): the gradients of rdx_qk_norm_rope at its inputs q and k, for incoming gradients
    dq_out and dk_out.  The weights' are float32 sums over all tokens and heads."""
    return (_module or _marshal()).qk_norm_rope_grad(q, k, q_weight, k_weight, positions, cos, sin, eps, interleaved,
                                                     dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, stream)


class KVCache:
    """A paged cache of 8-bit keys and values: codes k, v (int8 or float8_e4m3fn) [pages, heads, page_size, head_dim] and
    float32 scales k_scale, v_scale [pages, heads, page_size].  The tensors stay the caller's; this checks them and keeps
    them alive.  Each call takes their addresses and shapes as they are then, so their storage may move or be given back
    and brought in again; a call while it is away is refused.  The tensors themselves cannot be replaced."""

    __slots__ = ("_tensors",)

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 4 or k.dtype not in KV_FORMATS:
            raise TypeError(f"KVCache: k must be a 4-D CUDA tensor of dtype in {tuple(KV_FORMATS)}")
        if min(k.shape[1:]) < 1:
            raise ValueError(f"KVCache: heads, page_size and head_dim must be at least 1, got k of shape {tuple(k.shape)}")
        for what, x, dtype, shape in (("k", k, k.dtype, k.shape), ("v", v, k.dtype, k.shape),
                                      ("k_scale", k_scale, torch.float32, k.shape[:3]),
                                      ("v_scale", v_scale, torch.float32, k.shape[:3])):
            if not isinstance(x, torch.Tensor) or x.device != k.device or x.dtype != dtype:
                raise TypeError(f"KVCache: {what} must be a {dtype} tensor on {k.device}")
            if x.shape != shape or not x.is_contiguous():
                raise ValueError(f"KVCache: {what} must be contiguous with shape {tuple(shape)}, got {tuple(x.shape)}")
        self._tensors = (k, v, k_scale, v_scale)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    pages = property(lambda self: self.k.shape[0])
    heads = property(lambda self: self.k.shape[1])
    page_size = property(lambda self: self.k.shape[2])
    head_dim = property(lambda self: self.k.shape[3])

    @classmethod
    def zeros(cls, pages: int, page_size: int, heads: int, head_dim: int, dtype=torch.int8, device="cuda") -> "KVCache":
        """A new cache of zeros (int8 or float8_e4m3fn)."""
        k, v = (torch.zeros(pages, heads, page_size, head_dim, dtype=torch.uint8, device=device).view(dtype)
                for _ in range(2))
        k_scale, v_scale = (torch.zeros(pages, heads, page_size, device=device) for _ in range(2))
        return cls(k, v, k_scale, v_scale)


def rdx_kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantises the rows of k and v [tokens, heads, head_dim] (float32 or bfloat16) into the cache, token t at slot
    slots[t] = page * page_size + offset (int64, all different; a slot outside the cache, such as -1, is skipped)."""
    (_module or _marshal()).kv_write(cache, k, v, slots, stream)


def rdx_kv_read(cache: KVCache, slots: torch.Tensor, dtype=torch.bfloat16, k_out: torch.Tensor | None = None,
                v_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, heads, head_dim] of `dtype`: the cache's rows at these slots as the values they stand for
    (zeros for a negative slot, NaN for one past the end)."""
    code = TYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"rdx_kv_read: expected dtype in {tuple(TYPE_CODES)}, got {dtype}")
    return (_module or _marshal()).kv_read(cache, slots, code, k_out, v_out, stream)


def rdx_kv_attend(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lens: torch.Tensor,
                  scale: float | None = None, max_len: int | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [batch, q_heads, head_dim]: attention of one query token a sequence, q (float32 or bfloat16), over the first
    lens[b] (int32) tokens of the cache's pages block_table[b] (int32 [batch, pages]).  scale: default head_dim ** -0.5.
    max_len: no length is above it (default: all the table's pages; a close bound lets few, short sequences take a
    faster way).  lse: a float32 [batch, q_heads] tensor that receives the logarithm of each softmax sum.  A sequence of
    length 0 gives zeros (lse -inf); a length outside [0, max_len] or a page outside the cache gives NaN.  The result is
    detached, like a reduction's: this operator, the cache's write and its read have no gradients."""
    return (_module or _marshal()).kv_attend(q, cache, block_table, lens, scale, max_len, out, lse, workspace, stream)


def rdx_kv_attend_workspace_bytes(cache: KVCache, batch: int, q_heads: int, max_len: int,
                                  dtype: torch.dtype | None = None) -> int:
    """Bytes of the workspace an rdx_kv_attend call of these sizes needs with a q of `dtype` (0: none).  The types need
    different sizes; dtype None: enough for each of them."""
    if dtype is not None and dtype not in TYPE_CODES:
        raise TypeError(f"rdx_kv_attend_workspace_bytes: expected dtype in {tuple(TYPE_CODES)}, got {dtype}")
    pages = -(-max_len // cache.page_size)
    return max(int(load().rdx_kv_attend_workspace_bytes(_KV_ATTEND_ARGS.pack(
        0, 0, 0, 0, cache.pages, cache.page_size, cache.heads, cache.head_dim, KV_FORMATS[cache.k.dtype], *(0,) * 6,
        0, 0, 0, 0, 0, batch, 0, pages, max_len, q_heads, code, 1.0)))
        for code in (TYPE_CODES.values() if dtype is None else (TYPE_CODES[dtype],)))
