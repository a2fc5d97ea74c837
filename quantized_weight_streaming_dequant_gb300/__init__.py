"""Python binding of the rf C ABI (include/rf.h): argument marshalling only.

Every computation runs in the CUDA kernels of ``_lib/librf.so``; this module
turns torch tensors into pointers and stream handles, allocates outputs with
torch (device memory is plumbing), and raises ``RFError`` on any non-OK
status.  There is no CPU fallback: if the library is missing or no GPU is
present, calls fail loudly.
"""
from __future__ import annotations

import ctypes
import re
from pathlib import Path

PKG = Path(__file__).resolve().parent
SO = PKG / "_lib" / "librf.so"
HEADER = PKG.parent / "include" / "rf.h"

Q4_0, Q8_0, Q4_K, Q6_K, MXFP4 = 2, 8, 12, 14, 39
FORMATS = {"Q4_0": Q4_0, "Q8_0": Q8_0, "Q4_K": Q4_K, "Q6_K": Q6_K, "MXFP4": MXFP4}
BLOCK_BYTES = {Q4_0: 18, Q8_0: 34, Q4_K: 144, Q6_K: 210, MXFP4: 17}
BLOCK_ELEMS = {Q4_0: 32, Q8_0: 32, Q4_K: 256, Q6_K: 256, MXFP4: 32}

F32, F16, BF16 = 0, 1, 30           # activation types
Y_F32 = 256                         # added to a product's: fp32 outputs
ROPE_HALF, ROPE_PAIRS = 0, 1        # rotation styles
ACT_NONE, ACT_SILU, ACT_GELU, ACT_SWIGLU, ACT_SWIGLU_CLAMPED = 0, 1, 2, 3, 4   # activations of rf_epilogue
KV_BLOCK = 32                       # tokens that share a scale byte of the KV cache

OK = 0
CHAIN = 1   # RF_CHAIN launch flag
STATUS = {0: "RF_OK", 1: "RF_ERR_INVALID_ARG", 2: "RF_ERR_UNSUPPORTED_FMT",
          3: "RF_ERR_NOT_PINNED", 4: "RF_ERR_ARENA_TOO_SMALL", 5: "RF_ERR_CUDA",
          6: "RF_ERR_TIMEOUT", 7: "RF_ERR_OOM", 8: "RF_ERR_MISALIGNED", 9: "RF_ERR_TOO_LARGE"}


class RFError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class Window(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("row_start", ctypes.c_int64),
                ("row_end", ctypes.c_int64), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class StreamStats(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64), ("blocks", ctypes.c_uint64),
                ("bytes_copied", ctypes.c_uint64), ("peak_bytes", ctypes.c_uint64),
                ("slot_bytes", ctypes.c_uint64), ("arena_bytes", ctypes.c_uint64),
                ("slots", ctypes.c_int32), ("last_block_rows", ctypes.c_int32)]


class ExpertCacheStats(ctypes.Structure):
    _fields_ = [("lookups", ctypes.c_uint64), ("hits", ctypes.c_uint64),
                ("fills", ctypes.c_uint64), ("bypasses", ctypes.c_uint64),
                ("evictions", ctypes.c_uint64), ("bytes_streamed", ctypes.c_uint64),
                ("bytes_cached", ctypes.c_uint64), ("slots", ctypes.c_int32),
                ("used", ctypes.c_int32)]


class KVCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class KVBatchStruct(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("past", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("table_width", ctypes.c_int32), ("n_seq", ctypes.c_int32),
                ("n_tok", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AttentionPlan(ctypes.Structure):
    _fields_ = [("part_positions", ctypes.c_int64), ("tiles", ctypes.c_int32), ("parts", ctypes.c_int32),
                ("item_tokens", ctypes.c_int32), ("head_tiles", ctypes.c_int32), ("sms", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("up_bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ld_residual", ctypes.c_int64), ("act", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("limit", ctypes.c_float), ("reserved", ctypes.c_int32)]


_P, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "rf_status_str": ([_I], ctypes.c_char_p),
    "rf_version": ([], _I),
    "rf_block_bytes": ([_I], _SZ),
    "rf_row_bytes": ([_I, _I64], _SZ),
    "rf_max_in_dim": ([_I, _I], _I64),
    "rf_dequantize": ([_I, _P, _I64, _P, _P], _I),
    "rf_gemv": ([_I, _P, _I64, _I64, _I64, _P, _P, _P], _I),
    "rf_gemv_batch": ([_I, _I64, _I, ctypes.POINTER(Window), _P], _I),
    "rf_gemv_ex": ([_I, _P, _I64, _I64, _I64, _P, _P, ctypes.c_uint, _P], _I),
    "rf_gemv_batch_ex": ([_I, _I64, _I, ctypes.POINTER(Window), ctypes.c_uint, _P], _I),
    "rf_ffn_swiglu_ex": ([_I, _P, _P, _P, _I64, _I64, _P, _P, _P, ctypes.c_uint, _P], _I),
    "rf_swiglu": ([_P, _P, _P, _I64, _P], _I),
    "rf_gelu": ([_P, _P, _I64, _P], _I),
    "rf_ffn_swiglu": ([_I, _P, _P, _P, _I64, _I64, _P, _P, _P, _P], _I),
    "rf_ffn_workspace_bytes": ([_I64], _SZ),
    "rf_gemv_host": ([_I, _P, _I64, _I64, _I64, _P, _P, _P], _I),
    "rf_gemm": ([_I, _P, _I64, _I64, _I64, _I, _P, _I64, _P, _I64, _P, _SZ, _P], _I),
    "rf_gemm_workspace_bytes": ([_I, _I64, _I], _SZ),
    "rf_gemv_multi": ([_I, _P, _I64, _I64, _I64, _I, _P, _I64, _P, _I64, ctypes.c_uint, _P], _I),
    "rf_ffn_swiglu_ws": ([_I, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, ctypes.c_uint, _P], _I),
    "rf_arena_create": ([_SZ, _I, ctypes.POINTER(_P)], _I),
    "rf_arena_destroy": ([_P], None),
    "rf_arena_wait": ([_P, _I], _I),
    "rf_arena_inject_fault": ([_P, _I, _I64, _I], _I),
    "rf_arena_configure": ([_P, _I, _I], _I),
    "rf_stream_plan": ([_I, _I64, _I64, _I64, _I, _SZ, ctypes.POINTER(_I64),
                        ctypes.POINTER(_I64), ctypes.POINTER(_SZ)], _I),
    "rf_stream_linear": ([_I, _P, _I64, _I64, _I64, _I64, _I, _P, _P, _P, _P], _I),
    "rf_stream_stats": ([_P, ctypes.POINTER(StreamStats)], _I),
    "rf_moe_route": ([_P, _I, _I, _P, _P, _P], _I),
    "rf_moe_workspace_bytes": ([_I, _I64, _I64, _I64], _SZ),
    "rf_moe_ffn": ([_I, _P, _I, _I, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P], _I),
    "rf_moe_ffn_biased": ([_I, _P, _I, _I, _P, _P, _P, _P, _P, _P, ctypes.c_float,
                           ctypes.c_float, _I64, _I64, _I64, _P, _P, _P, _P], _I),
    "rf_moe_ffn_noalloc": ([_I, _P, _I, _I, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P], _I),
    "rf_moe_ffn_host": ([_I, _P, _I, _I, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P], _I),
    "rf_expert_cache_create": ([_I, _I64, _I64, _I, ctypes.POINTER(_P)], _I),
    "rf_expert_cache_destroy": ([_P], None),
    "rf_expert_cache_stats": ([_P, ctypes.POINTER(ExpertCacheStats)], _I),
    "rf_moe_ffn_streamed": ([_I, _P, _I, _I, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P,
                             _P], _I),
    "rf_norm_residual": ([_I, _I64, _I64, _P, _I64, _P, _P, _I64, ctypes.c_float, _P, _I64, _P, _I64,
                          _P, _P, _I64, ctypes.c_float, ctypes.c_uint, _P], _I),
    "rf_kv_append": ([_P, _P, _I, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64,
                      _I, _P, _P, _I64, _I, _I, ctypes.c_uint, _P], _I),
    "rf_kv_read": ([_P, _P, _P, _P, ctypes.c_uint, _P], _I),
    "rf_attention": ([_P, _P, _I, _P, _I64, _I64, _I, ctypes.c_float, _I64, _P, _P, _I64, _I64,
                      _I64, _P, _SZ, ctypes.c_uint, _P], _I),
    "rf_attention_workspace_bytes": ([_P, _P, _I, _I, _I64, _I64], _SZ),
    "rf_gemm_fused": ([_I, _P, _P, _I64, _I64, _I64, _I, _I64, _P, _I64, _P, _P, _I64, _P, _SZ, _P], _I),
    "rf_gemm_fused_workspace_bytes": ([_I, _I64, _I64, _I, _I64], _SZ),
    "rf_gemm_grouped": ([_I, _P, _P, _I, _I64, _I64, _I, _P, _I64, _I64, _P, _P, _I, _I64, _P, _P, _I64, _P,
                         _SZ, _P], _I),
    "rf_gemm_grouped_workspace_bytes": ([_I, _I, _I64, _I64, _I, _I64], _SZ),
    "rf_moe_route_tokens": ([_I, _P, _I64, _I64, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "rf_moe_route_tokens_workspace_bytes": ([_I64, _I, _I], _SZ),
    "rf_moe_ffn_tokens": ([_I, _I, _I, _P, _I64, _I, _I, _I64, _P, _P, _P, _P, _P, _P, _I, ctypes.c_float,
                           ctypes.c_float, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _SZ, _P], _I),
    "rf_moe_tokens_workspace_bytes": ([_I, _I, _I, _I64, _I64, _I, _I64], _SZ),
    "rf_device_status": ([], _I),
    "rf_debug_arm_wait_fault": ([ctypes.c_uint32], _I),
    "rf_debug_attention_plan": ([_P, _P, _I, _I, _I64, _I64, ctypes.POINTER(AttentionPlan)], _I),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load librf.so (built by build.py); raises if it is missing."""
    global _lib
    if _lib is None:
        if not SO.exists():
            raise RuntimeError(f"{SO} is missing: build it with "
                               "`python -m quantized_weight_streaming_dequant_gb300.build`")
        L = ctypes.CDLL(str(SO))
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Names of the functions include/rf.h declares."""
    return re.findall(r"^RF_API[^(]*?\b(rf_\w+)\(", HEADER.read_text(), flags=re.M)


def _check(code: int, what: str) -> None:
    if code != OK:
        raise RFError(code, what)


_raw_stream = _current_device = None


def _stream(stream):
    global _raw_stream, _current_device
    if stream is None:
        if _raw_stream is None:
            # The handle alone: building a torch.cuda.Stream costs 3 us a call.
            import torch
            torch.cuda.init()
            _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_DTYPES = _empty = _empty_like = _F32_TYPE = _U8_TYPE = _I32_TYPE = None


def _look_up() -> None:
    """torch's names, once: an import statement in a function costs each call 0.5 us."""
    global _DTYPES, _empty, _empty_like, _F32_TYPE, _U8_TYPE, _I32_TYPE
    import torch
    _I32_TYPE = torch.int32
    _empty, _empty_like, _F32_TYPE, _U8_TYPE = torch.empty, torch.empty_like, torch.float32, torch.uint8
    _DTYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


def _new(stream, size, dtype, device, out: bool = True):
    """A device tensor for a call on `stream` (None: the current stream), from
    that stream's own memory, as torch's operators take theirs: memory of
    another stream may still be in use there, and may be handed on there while
    this call's kernels run.  out: the caller may also use it, and then drop it,
    on the current stream."""
    if _empty is None:
        _look_up()
    if stream is None or _stream(stream) == _stream(None):
        return _empty(size, dtype=dtype, device=device)
    import torch
    current = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = _empty(size, dtype=dtype, device=device)
    if out:
        t.record_stream(current)
    return t


def _new_f32(stream, size, like):
    """_new: float32, on the device of `like`."""
    if _empty is None:
        _look_up()
    return _new(stream, size, _F32_TYPE, like.device)


def _new_like(stream, like):
    """_new: contiguous, of the shape and type of `like`."""
    if _empty is None:
        _look_up()
    if stream is None and like.is_contiguous():
        return _empty_like(like)
    return _new(stream, like.shape, like.dtype, like.device)


def _dev_ptr(t, what: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def status_str(code: int) -> str:
    return lib().rf_status_str(code).decode()


def block_bytes(fmt: int) -> int:
    return lib().rf_block_bytes(fmt)


def row_bytes(fmt: int, in_dim: int) -> int:
    return lib().rf_row_bytes(fmt, in_dim)


def max_in_dim(fmt: int, n_x: int = 1) -> int:
    return lib().rf_max_in_dim(fmt, n_x)


def dequantize(fmt: int, W, n_blocks: int | None = None, out=None, stream=None):
    if n_blocks is None:
        n_blocks = W.numel() // BLOCK_BYTES[fmt]
    if out is None:
        out = _new_f32(stream, BLOCK_ELEMS[fmt] * n_blocks, W)
    _check(lib().rf_dequantize(fmt, _dev_ptr(W, "W"), n_blocks, _dev_ptr(out, "out"),
                               _stream(stream)), "rf_dequantize")
    return out


def gemv(fmt: int, W, row_start: int, row_end: int, in_dim: int, x, y=None, stream=None,
         flags: int = 0):
    if y is None:
        y = _new_f32(stream, max(row_end - row_start, 0), x)
    _check(lib().rf_gemv_ex(fmt, _dev_ptr(W, "W"), row_start, row_end, in_dim, _dev_ptr(x, "x"),
                            _dev_ptr(y, "y") if y.numel() else 1, flags, _stream(stream)),
           "rf_gemv")
    return y


def gemv_multi(fmt: int, W, row_start: int, row_end: int, in_dim: int, X, Y=None, stream=None,
               flags: int = 0):
    """rf_gemv_multi: X is (n_tok, in_dim) float32 on the device (rows may be
    strided); returns Y (n_tok, row_end - row_start)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit stride along in_dim")
    n_tok = X.shape[0]
    if Y is None:
        Y = _new_f32(stream, (n_tok, max(row_end - row_start, 0)), X)
    if Y.dim() != 2 or Y.stride(1) != 1:
        raise ValueError("Y must be 2-D with unit stride along the rows")
    _check(lib().rf_gemv_multi(fmt, _dev_ptr(W, "W"), row_start, row_end, in_dim, n_tok,
                               X.data_ptr(), X.stride(0), Y.data_ptr(), Y.stride(0), flags,
                               _stream(stream)), "rf_gemv_multi")
    return Y


def gemm_workspace_bytes(fmt: int, in_dim: int, n_tok: int) -> int:
    return int(lib().rf_gemm_workspace_bytes(fmt, in_dim, n_tok))


def gemm(fmt: int, W, row_start: int, row_end: int, in_dim: int, X, Y=None, workspace=None,
         stream=None):
    """rf_gemm (tensor cores): X is (n_tok, in_dim) float32 on the device
    (rows may be strided); returns Y (n_tok, row_end - row_start).  The
    workspace (a uint8 device tensor) is allocated when not given."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit stride along in_dim")
    n_tok = X.shape[0]
    if Y is None:
        Y = _new_f32(stream, (n_tok, max(row_end - row_start, 0)), X)
    if Y.dim() != 2 or Y.stride(1) != 1:
        raise ValueError("Y must be 2-D with unit stride along the rows")
    need = gemm_workspace_bytes(fmt, in_dim, n_tok)
    if workspace is None and need > 0:
        workspace = _new(stream, need, _U8_TYPE, X.device, out=False)
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    _check(lib().rf_gemm(fmt, _dev_ptr(W, "W"), row_start, row_end, in_dim, n_tok,
                         X.data_ptr(), X.stride(0), Y.data_ptr(), Y.stride(0), ws, ws_bytes,
                         _stream(stream)), "rf_gemm")
    return Y


def gemv_batch(fmt: int, in_dim: int, windows, stream=None, flags: int = 0):
    """windows: list of (W, row_start, row_end, x, y) with device tensors."""
    arr = (Window * max(len(windows), 1))()
    for i, (W, r0, r1, x, y) in enumerate(windows):
        arr[i] = Window(_dev_ptr(W, "W"), r0, r1, _dev_ptr(x, "x"), _dev_ptr(y, "y"))
    _check(lib().rf_gemv_batch_ex(fmt, in_dim, len(windows), arr, flags, _stream(stream)),
           "rf_gemv_batch")


def swiglu(g, u, h=None, stream=None):
    h = _new_like(stream, g) if h is None else h
    _check(lib().rf_swiglu(_dev_ptr(g, "g"), _dev_ptr(u, "u"), _dev_ptr(h, "h"), g.numel(),
                           _stream(stream)), "rf_swiglu")
    return h


def gelu(z, h=None, stream=None):
    h = _new_like(stream, z) if h is None else h
    _check(lib().rf_gelu(_dev_ptr(z, "z"), _dev_ptr(h, "h"), z.numel(), _stream(stream)),
           "rf_gelu")
    return h


def gemv_host(fmt: int, host_W, row_start: int, row_end: int, in_dim: int, x, y=None,
              stream=None):
    """rf_gemv_host: host_W is a page-locked CPU tensor (uint8) read in place."""
    if host_W.is_cuda or not host_W.is_contiguous():
        raise ValueError("host_W must be a contiguous CPU tensor")
    if y is None:
        y = _new_f32(stream, max(row_end - row_start, 0), x)
    _check(lib().rf_gemv_host(fmt, host_W.data_ptr(), row_start, row_end, in_dim,
                              _dev_ptr(x, "x"), _dev_ptr(y, "y") if y.numel() else 1,
                              _stream(stream)), "rf_gemv_host")
    return y


def ffn_workspace(n_ff: int, device):
    """Device workspace for ffn_swiglu's digit hand-off between its launches."""
    import torch
    return torch.empty(lib().rf_ffn_workspace_bytes(n_ff), dtype=torch.uint8, device=device)


def ffn_swiglu(fmt: int, gate, up, down, n_ff: int, n_embd: int, x, y=None, h=None,
               stream=None, flags: int = 0, workspace=None):
    """rf_ffn_swiglu_ws (workspace: from ffn_workspace, or None)."""
    y = _new_f32(stream, n_embd, x) if y is None else y
    h = _new_f32(stream, n_ff, x) if h is None else h
    _check(lib().rf_ffn_swiglu_ws(fmt, _dev_ptr(gate, "gate"), _dev_ptr(up, "up"),
                                  _dev_ptr(down, "down"), n_ff, n_embd, _dev_ptr(x, "x"),
                                  _dev_ptr(y, "y"), _dev_ptr(h, "h"),
                                  _dev_ptr(workspace, "workspace") if workspace is not None
                                  else None, flags, _stream(stream)),
           "rf_ffn_swiglu")
    return y, h


def stream_plan(fmt: int, in_dim: int, n_rows: int, block_rows: int, depth: int,
                arena_bytes: int):
    """(effective rows per block, blocks, peak arena bytes); host only."""
    eff, nblk, peak = _I64(0), _I64(0), _SZ(0)
    _check(lib().rf_stream_plan(fmt, in_dim, n_rows, block_rows, depth, arena_bytes,
                                ctypes.byref(eff), ctypes.byref(nblk), ctypes.byref(peak)),
           "rf_stream_plan")
    return eff.value, nblk.value, peak.value


FAULT_NONE, FAULT_COPY_FAIL, FAULT_COPY_STALL = 0, 1, 2
ARENA_MERGE_RUNS, ARENA_LANES = 1, 2


class Arena:
    """Bounded device arena with its copy stream (rf_arena_create); device -1
    = the current device."""

    def __init__(self, nbytes: int, device: int = -1):
        h = _P()
        _check(lib().rf_arena_create(nbytes, device, ctypes.byref(h)), "rf_arena_create")
        self.handle = h
        self.nbytes = nbytes

    def wait(self, timeout_ms: int) -> int:
        """rf_arena_wait: the status (OK, or TIMEOUT while work is outstanding)."""
        code = lib().rf_arena_wait(self.handle, timeout_ms)
        if code not in (OK, 6):
            raise RFError(code, "rf_arena_wait")
        return code

    def configure(self, option: int, value: bool) -> None:
        """rf_arena_configure: ARENA_MERGE_RUNS / ARENA_LANES on or off."""
        _check(lib().rf_arena_configure(self.handle, option, int(bool(value))),
               "rf_arena_configure")

    def inject_fault(self, kind: int, block: int, ms: int = 0) -> None:
        """rf_arena_inject_fault (test hook)."""
        _check(lib().rf_arena_inject_fault(self.handle, kind, block, ms), "rf_arena_inject_fault")

    def close(self) -> None:
        if self.handle is not None and self.handle.value:
            lib().rf_arena_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stream_linear(self, fmt: int, host_W, in_dim: int, row_start: int, row_end: int,
                      block_rows: int, depth: int, x, y=None, stream=None):
        """host_W: page-locked CPU tensor (uint8) holding row 0 onwards."""
        if host_W.is_cuda or not host_W.is_contiguous():
            raise ValueError("host_W must be a contiguous CPU tensor")
        if y is None:
            y = _new_f32(stream, max(row_end - row_start, 0), x)
        _check(lib().rf_stream_linear(fmt, host_W.data_ptr(), in_dim, row_start, row_end,
                                      block_rows, depth, self.handle, _dev_ptr(x, "x"),
                                      _dev_ptr(y, "y") if y.numel() else 1, _stream(stream)),
               "rf_stream_linear")
        return y

    def stats(self) -> dict:
        s = StreamStats()
        _check(lib().rf_stream_stats(self.handle, ctypes.byref(s)), "rf_stream_stats")
        return {k: getattr(s, k) for k, _ in StreamStats._fields_}


class ExpertCache:
    """Device cache of whole experts (rf_expert_cache_create)."""

    def __init__(self, fmt: int, n_ff: int, n_embd: int, slots: int):
        h = _P()
        _check(lib().rf_expert_cache_create(fmt, n_ff, n_embd, slots, ctypes.byref(h)),
               "rf_expert_cache_create")
        self.handle = h

    def close(self) -> None:
        if self.handle is not None and self.handle.value:
            lib().rf_expert_cache_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self) -> dict:
        s = ExpertCacheStats()
        _check(lib().rf_expert_cache_stats(self.handle, ctypes.byref(s)),
               "rf_expert_cache_stats")
        return {k: getattr(s, k) for k, _ in ExpertCacheStats._fields_}


def moe_ffn_streamed(fmt: int, logits, top_k: int, host_gate, host_up, host_down, n_ff: int,
                     n_embd: int, block_rows: int, depth: int, arena: "Arena", x, cache=None,
                     y=None, workspace=None, stream=None):
    """rf_moe_ffn_streamed: experts in page-locked CPU tensors, one layer-wide
    prefetch plan through `arena`, an optional ExpertCache."""
    for t, nm in ((host_gate, "host_gate"), (host_up, "host_up"), (host_down, "host_down")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous CPU tensor")
    y = _new_f32(stream, n_embd, x) if y is None else y
    if workspace is None:
        workspace = moe_workspace(top_k, n_ff, n_embd, block_rows, x.device, stream)
    _check(lib().rf_moe_ffn_streamed(fmt, _dev_ptr(logits, "logits"), logits.numel(), top_k,
                                     host_gate.data_ptr(), host_up.data_ptr(),
                                     host_down.data_ptr(), n_ff, n_embd, block_rows, depth,
                                     arena.handle, cache.handle if cache is not None else None,
                                     _dev_ptr(x, "x"), _dev_ptr(y, "y"),
                                     _dev_ptr(workspace, "workspace"), _stream(stream)),
           "rf_moe_ffn_streamed")
    return y, workspace


def moe_route(logits, top_k: int, stream=None):
    import torch
    idx = _new(stream, top_k, torch.int32, logits.device)
    w = _new_f32(stream, top_k, logits)
    _check(lib().rf_moe_route(_dev_ptr(logits, "logits"), logits.numel(), top_k,
                              _dev_ptr(idx, "idx"), _dev_ptr(w, "w"), _stream(stream)),
           "rf_moe_route")
    return idx, w


def moe_workspace_bytes(top_k: int, n_ff: int, n_embd: int, block_rows: int) -> int:
    return lib().rf_moe_workspace_bytes(top_k, n_ff, n_embd, block_rows)


def moe_workspace(top_k: int, n_ff: int, n_embd: int, block_rows: int, device, stream=None):
    if _empty is None:
        _look_up()
    return _new(stream, moe_workspace_bytes(top_k, n_ff, n_embd, block_rows), _U8_TYPE, device)


def moe_ffn(fmt: int, logits, top_k: int, gate, up, down, n_ff: int, n_embd: int,
            block_rows: int, x, y=None, workspace=None, stream=None):
    y = _new_f32(stream, n_embd, x) if y is None else y
    if workspace is None:
        workspace = moe_workspace(top_k, n_ff, n_embd, block_rows, x.device, stream)
    _check(lib().rf_moe_ffn(fmt, _dev_ptr(logits, "logits"), logits.numel(), top_k,
                            _dev_ptr(gate, "gate"), _dev_ptr(up, "up"), _dev_ptr(down, "down"),
                            n_ff, n_embd, block_rows, _dev_ptr(x, "x"), _dev_ptr(y, "y"),
                            _dev_ptr(workspace, "workspace"), _stream(stream)), "rf_moe_ffn")
    return y, workspace


def moe_ffn_biased(fmt: int, logits, top_k: int, gate, up, down, gate_bias, up_bias, down_bias,
                   alpha: float, limit: float, n_ff: int, n_embd: int, block_rows: int, x,
                   y=None, workspace=None, stream=None):
    """rf_moe_ffn_biased: biases are device float32 tensors (or None)."""
    y = _new_f32(stream, n_embd, x) if y is None else y
    if workspace is None:
        workspace = moe_workspace(top_k, n_ff, n_embd, block_rows, x.device, stream)
    opt = lambda t, nm: None if t is None else _dev_ptr(t, nm)   # noqa: E731
    _check(lib().rf_moe_ffn_biased(fmt, _dev_ptr(logits, "logits"), logits.numel(), top_k,
                                   _dev_ptr(gate, "gate"), _dev_ptr(up, "up"),
                                   _dev_ptr(down, "down"), opt(gate_bias, "gate_bias"),
                                   opt(up_bias, "up_bias"), opt(down_bias, "down_bias"),
                                   alpha, limit, n_ff, n_embd, block_rows, _dev_ptr(x, "x"),
                                   _dev_ptr(y, "y"), _dev_ptr(workspace, "workspace"),
                                   _stream(stream)), "rf_moe_ffn_biased")
    return y, workspace


def moe_ffn_noalloc(fmt: int, logits, top_k: int, gate, up, down, n_ff: int, n_embd: int,
                    block_rows: int, x, y, stream=None):
    """rf_moe_ffn_noalloc: the library's own fixed scratch instead of a
    workspace; y must be preallocated."""
    _check(lib().rf_moe_ffn_noalloc(fmt, _dev_ptr(logits, "logits"), logits.numel(), top_k,
                                    _dev_ptr(gate, "gate"), _dev_ptr(up, "up"),
                                    _dev_ptr(down, "down"), n_ff, n_embd, block_rows,
                                    _dev_ptr(x, "x"), _dev_ptr(y, "y"), _stream(stream)),
           "rf_moe_ffn_noalloc")
    return y


def moe_ffn_host(fmt: int, logits, top_k: int, gate, up, down, n_ff: int, n_embd: int,
                 block_rows: int, x, y=None, workspace=None, stream=None):
    """rf_moe_ffn_host: gate/up/down are page-locked CPU tensors read in place."""
    for t in (gate, up, down):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("expert tensors must be contiguous CPU tensors")
    y = _new_f32(stream, n_embd, x) if y is None else y
    if workspace is None:
        workspace = moe_workspace(top_k, n_ff, n_embd, block_rows, x.device, stream)
    _check(lib().rf_moe_ffn_host(fmt, _dev_ptr(logits, "logits"), logits.numel(), top_k,
                                 gate.data_ptr(), up.data_ptr(), down.data_ptr(), n_ff, n_embd,
                                 block_rows, _dev_ptr(x, "x"), _dev_ptr(y, "y"),
                                 _dev_ptr(workspace, "workspace"), _stream(stream)),
           "rf_moe_ffn_host")
    return y, workspace


def moe_workspace_views(workspace, top_k: int, n_ff: int):
    """(idx, w, h) views into an rf_moe_ffn workspace (for inspection)."""
    import torch
    idx = workspace[:32].view(torch.int32)[:top_k]
    w = workspace[256:288].view(torch.float32)[:top_k]
    h = workspace[512:512 + 4 * top_k * n_ff].view(torch.float32).view(top_k, n_ff)
    return idx, w, h


def _dtype(t) -> int:
    """The activation type of a tensor."""
    if _DTYPES is None:
        _look_up()
    d = _DTYPES.get(t.dtype)   # F32 is 0
    if d is None:
        raise ValueError(f"activations are float32, float16 or bfloat16, not {t.dtype}")
    return d


def _f32_ptr(t, n: int, what: str):
    """Data pointer of n contiguous float32 device values, or None."""
    if t is None:
        return None
    if not t.is_cuda or _dtype(t) != F32 or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what} must be {n} contiguous float32 values on the device")
    return t.data_ptr()


def _rows(t, n_tok: int, n: int, dtype: int, what: str):
    """(pointer, row stride) of a (n_tok, n) tensor with contiguous rows; (None, 0) for None."""
    if t is None:
        return None, 0
    if not t.is_cuda or _dtype(t) != dtype or t.shape != (n_tok, n):
        raise ValueError(f"{what} must be a ({n_tok}, {n}) CUDA tensor of the call's type")
    ld, one = t.stride()
    if one != 1 and n > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), ld if n_tok > 1 or ld > n else n   # the stride of one row says nothing


def norm_residual(residual, x=None, *, post_weight=None, gate=None, scale: float = 1.0, weight=None,
                  eps: float = 1e-5, residual_out=None, y=None, norm: bool = True, stream=None,
                  flags: int = 0):
    """rf_norm_residual: residual and x are (n_tok, n) (rows may be strided;
    either may be None); gate is (n,) or (n_tok, n) float32.  Returns
    (residual + scale * gate * post_norm(x), its norm); the norm is None with
    norm=False."""
    like = residual if residual is not None else x
    if like is None or like.dim() != 2:
        raise ValueError("residual or x must be given, (n_tok, n)")
    n_tok, n = like.shape
    dt = _dtype(like)
    px, ldx = _rows(x, n_tok, n, dt, "x")
    pr, ldr = _rows(residual, n_tok, n, dt, "residual")
    if residual_out is None:
        residual_out = _new_like(stream, like)
        po, ldo = residual_out.data_ptr(), n
    else:
        po, ldo = _rows(residual_out, n_tok, n, dt, "residual_out")
    if y is None and norm:
        y = _new_like(stream, like)
        py, ldy = y.data_ptr(), n
    else:
        py, ldy = _rows(y, n_tok, n, dt, "y")
    pg, ldg = None, 0
    if gate is not None:
        pg, ldg = _rows(gate, n_tok, n, F32, "gate") if gate.dim() == 2 else (_f32_ptr(gate, n, "gate"), 0)
    _check(lib().rf_norm_residual(dt, n_tok, n, px, ldx, _f32_ptr(post_weight, n, "post_weight"), pg, ldg,
                                  scale, pr, ldr, po, ldo, _f32_ptr(weight, n, "weight"), py, ldy, eps,
                                  flags, _stream(stream)), "rf_norm_residual")
    return residual_out, y


class KVCache:
    """A paged KV cache over the caller's tensors: k, v int8 (n_pages,
    n_kv_heads, page_size, head_dim) and k_scale, v_scale uint8 (n_pages,
    n_kv_heads, page_size / 32)."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        _look_up()
        if k.dim() != 4 or v.shape != k.shape or k.dtype != torch.int8 or v.dtype != torch.int8:
            raise ValueError("k and v must be int8, (n_pages, n_kv_heads, page_size, head_dim)")
        n_pages, n_kv, page, dim = k.shape
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.uint8 or tuple(t.shape) != (n_pages, n_kv, page // KV_BLOCK):
                raise ValueError(f"{what} must be uint8, (n_pages, n_kv_heads, page_size / {KV_BLOCK})")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n_pages, n_kv, page, dim
        self.device = k.device
        self.struct = KVCacheStruct(_dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(k_scale, "k_scale"),
                                    _dev_ptr(v_scale, "v_scale"), n_pages, page, n_kv, dim, 0)
        self.ref = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, device="cuda"):
        import torch
        codes = (n_pages, n_kv_heads, page_size, head_dim)
        scales = (n_pages, n_kv_heads, page_size // KV_BLOCK)
        return cls(torch.zeros(codes, dtype=torch.int8, device=device),
                   torch.zeros(codes, dtype=torch.int8, device=device),
                   torch.zeros(scales, dtype=torch.uint8, device=device),
                   torch.zeros(scales, dtype=torch.uint8, device=device))


class KVBatch:
    """The tokens of one call (rf_kv_batch): page_table (n_seq, width), past
    (n_seq,) and q_start (n_seq + 1,) are int32 device tensors that the
    kernels read at run time; n_tok is the number of rows of the call."""

    def __init__(self, page_table, past, q_start, n_tok: int):
        import torch
        n_seq = past.numel()
        for t, what in ((page_table, "page_table"), (past, "past"), (q_start, "q_start")):
            if not t.is_cuda or t.dtype != torch.int32 or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise ValueError(f"{what} must be an int32 CUDA tensor, its last dimension contiguous")
        if page_table.dim() != 2 or page_table.shape[0] != n_seq or past.dim() != 1 or \
                q_start.dim() != 1 or q_start.numel() != n_seq + 1:
            raise ValueError("page_table is (n_seq, width), past (n_seq,), q_start (n_seq + 1,)")
        self.page_table, self.past, self.q_start = page_table, past, q_start
        self.n_seq, self.n_tok, self.width = n_seq, n_tok, page_table.shape[1]
        stride = max(page_table.stride(0), self.width) if n_seq == 1 else page_table.stride(0)
        self.struct = KVBatchStruct(page_table.data_ptr(), past.data_ptr(), q_start.data_ptr(),
                                    stride, self.width, n_seq, n_tok, 0)
        self.ref = ctypes.addressof(self.struct)


def _heads(t, n_tok: int, dim: int, dtype: int, what: str):
    """(pointer, token stride, head stride, heads) of a (n_tok, heads, dim) tensor."""
    if not t.is_cuda or _dtype(t) != dtype or t.dim() != 3:
        raise ValueError(f"{what} must be a ({n_tok}, heads, {dim}) CUDA tensor of the call's type")
    nt, heads, d = t.shape
    lt, lh, one = t.stride()
    if nt != n_tok or d != dim or one != 1:
        raise ValueError(f"{what} must be ({n_tok}, heads, {dim}), the last dimension contiguous")
    # strides of dimensions of one element say nothing
    return t.data_ptr(), lt if nt > 1 or lt > dim else dim, lh if heads > 1 or lh > dim else dim, heads


def kv_append(cache: KVCache, batch: KVBatch, k, v, q=None, q_out=None, cos=None, sin=None,
              rope: int = ROPE_HALF, stream=None, flags: int = 0):
    """rf_kv_append: k, v (n_tok, n_kv_heads, head_dim) go to the cache, rotated
    (k) by the tables cos, sin (n_pos, rot / 2); returns the rotated q
    (n_tok, n_heads, head_dim), or None without q."""
    n_tok, dim, dt = batch.n_tok, cache.head_dim, _dtype(k)
    pk, klt, klh, kh = _heads(k, n_tok, dim, dt, "k")
    pv, vlt, vlh, vh = _heads(v, n_tok, dim, dt, "v")
    if kh != cache.n_kv_heads or vh != kh:
        raise ValueError("k and v must have the cache's heads")
    pq = po = None
    qlt = qlh = olt = olh = nh = 0
    if q is not None:
        pq, qlt, qlh, nh = _heads(q, n_tok, dim, dt, "q")
        if q_out is None:
            q_out = _new_like(stream, q)
            po, olt, olh = q_out.data_ptr(), nh * dim, dim
        else:
            po, olt, olh, oh = _heads(q_out, n_tok, dim, dt, "q_out")
            if oh != nh:
                raise ValueError("q_out must be like q")
    pc = ps = None
    n_pos = rot = 0
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be two (n_pos, rot / 2) tables")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        pc, ps = _f32_ptr(cos, cos.numel(), "cos"), _f32_ptr(sin, cos.numel(), "sin")
    _check(lib().rf_kv_append(cache.ref, batch.ref, dt, pk, klt, klh, pv, vlt, vlh, pq, qlt, qlh,
                              po, olt, olh, nh, pc, ps, n_pos, rot, rope, flags, _stream(stream)),
           "rf_kv_append")
    return q_out


def kv_read(cache: KVCache, batch: KVBatch, k_out=None, v_out=None, stream=None, flags: int = 0):
    """rf_kv_read: the cache's values at the batch's positions, two float32
    tensors (n_tok, n_kv_heads, head_dim)."""
    shape = (batch.n_tok, cache.n_kv_heads, cache.head_dim)
    n = shape[0] * shape[1] * shape[2]
    if k_out is None:
        k_out = _new(stream, shape, _F32_TYPE, cache.device)
    if v_out is None:
        v_out = _new(stream, shape, _F32_TYPE, cache.device)
    pk, pv = _f32_ptr(k_out, n, "k_out"), _f32_ptr(v_out, n, "v_out")
    _check(lib().rf_kv_read(cache.ref, batch.ref, pk, pv, flags, _stream(stream)), "rf_kv_read")
    return k_out, v_out


def attention_workspace(cache: KVCache, batch: KVBatch, q, max_len: int = 0, window: int = 0, stream=None):
    """Device workspace for attention() with these arguments on `stream`, or None."""
    n = lib().rf_attention_workspace_bytes(cache.ref, batch.ref, _dtype(q), q.shape[1], window, max_len)
    return _new(stream, n, _U8_TYPE, q.device, out=False) if n else None


def attention(cache: KVCache, batch: KVBatch, q, out=None, scale: float | None = None, window: int = 0,
              sinks=None, max_len: int = 0, workspace=None, stream=None, flags: int = 0):
    """rf_attention: q (n_tok, n_heads, head_dim) against the cache, which
    already holds the batch's own tokens; scale defaults to head_dim ** -0.5.
    The workspace is allocated when not given."""
    n_tok, dim, dt = batch.n_tok, cache.head_dim, _dtype(q)
    pq, qlt, qlh, nh = _heads(q, n_tok, dim, dt, "q")
    if out is None:
        out = _new_like(stream, q)
        po, olt, olh = out.data_ptr(), nh * dim, dim
    else:
        po, olt, olh, oh = _heads(out, n_tok, dim, dt, "out")
        if oh != nh:
            raise ValueError("out must be like q")
    if workspace is None:
        workspace = attention_workspace(cache, batch, q, max_len, window, stream)
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    _check(lib().rf_attention(cache.ref, batch.ref, dt, pq, qlt, qlh, nh,
                              dim ** -0.5 if scale is None else scale, window,
                              _f32_ptr(sinks, nh, "sinks"), po, olt, olh, max_len, ws, ws_bytes, flags,
                              _stream(stream)), "rf_attention")
    return out


def _matrix_rows(t, what: str):
    """(pointer, row stride, rows, columns, type) of a 2-D CUDA tensor with contiguous rows."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    n_tok, n = t.shape
    ld, one = t.stride()
    if one != 1 and n > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), ld if n_tok > 1 or ld > n else n, n_tok, n, _dtype(t)


def _weights(t, rows: int, fmt: int, in_dim: int, what: str) -> int:
    """Data pointer of a stack of `rows` quantized rows (uint8, contiguous)."""
    p = _dev_ptr(t, what)
    if t.numel() * t.element_size() < rows * (in_dim // BLOCK_ELEMS[fmt]) * BLOCK_BYTES[fmt]:
        raise ValueError(f"{what} is shorter than its {rows} rows")
    return p


def _known_fmt(fmt: int) -> int:
    if fmt not in BLOCK_BYTES:
        raise RFError(2, "weight format")
    return fmt


def _epilogue(n_bias, n_tok, rows, dt, act, up, bias, up_bias, alpha, limit, residual):
    pr, ldr = _rows(residual, n_tok, rows, dt, "residual")
    return Epilogue(_f32_ptr(bias, n_bias, "bias"), _f32_ptr(up_bias, n_bias, "up_bias"), pr, ldr, act, alpha, limit, 0)


def _space(workspace, need: int, stream, device):
    """(tensor, pointer, bytes) of a workspace, allocated when not given."""
    if workspace is None and need > 0:
        if _empty is None:
            _look_up()
        workspace = _new(stream, need, _U8_TYPE, device, out=False)
    if workspace is None:
        return None, None, 0
    return workspace, _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _product_types(dt: int, y_f32: bool):
    """(dtype of a product of X's type, Y's type)"""
    return (dt | Y_F32, F32) if y_f32 else (dt, dt)


def gemm_fused_workspace(fmt: int, rows: int, in_dim: int, X, stream=None, y_f32: bool = False):
    """Device workspace for gemm_fused() of X on `stream`, or None."""
    n = lib().rf_gemm_fused_workspace_bytes(fmt, rows, in_dim, _product_types(_dtype(X), y_f32)[0], X.shape[0])
    return _new(stream, n, _U8_TYPE, X.device, out=False) if n else None


def gemm_fused(fmt: int, W, row_start: int, row_end: int, in_dim: int, X, Y=None, *, act: int = ACT_NONE, up=None,
               bias=None, up_bias=None, alpha: float = 1.702, limit: float = 7.0, residual=None, workspace=None,
               stream=None, y_f32: bool = False):
    """rf_gemm_fused: residual + act(W X + bias, up X + up_bias) for the rows
    [row_start, row_end).  X (n_tok, in_dim) and residual (n_tok, rows) are of
    one type (rows may be strided); biases are float32, one per row of the
    window.  Returns Y (n_tok, rows), of X's type; with y_f32 Y and residual
    are float32."""
    _known_fmt(fmt)
    px, ldx, n_tok, n, dt = _matrix_rows(X, "X")
    if n != in_dim:
        raise ValueError(f"X must be (n_tok, {in_dim})")
    rows = max(row_end - row_start, 0)
    dt, dty = _product_types(dt, y_f32)
    if Y is None:
        Y = _new(stream, (n_tok, rows), _F32_TYPE if y_f32 else X.dtype, X.device)
    py, ldy = _rows(Y, n_tok, rows, dty, "Y")
    e = _epilogue(rows, n_tok, rows, dty, act, up, bias, up_bias, alpha, limit, residual)
    if workspace is None:
        need = lib().rf_gemm_fused_workspace_bytes(fmt, rows, in_dim, dt, n_tok)
    workspace, ws, ws_bytes = _space(workspace, need if workspace is None else 0, stream, X.device)
    _check(lib().rf_gemm_fused(fmt, _weights(W, max(row_end, 0), fmt, in_dim, "W"),
                               None if up is None else _weights(up, max(row_end, 0), fmt, in_dim, "up"), row_start,
                               row_end, in_dim, dt, n_tok, px, ldx, ctypes.byref(e), py, ldy, ws, ws_bytes,
                               _stream(stream)), "rf_gemm_fused")
    return Y


def gemm_grouped_workspace(fmt: int, n_group: int, rows: int, in_dim: int, X, n_row: int, stream=None,
                           y_f32: bool = False):
    """Device workspace for gemm_grouped() of n_row rows on `stream`, or None."""
    n = lib().rf_gemm_grouped_workspace_bytes(fmt, n_group, rows, in_dim, _product_types(_dtype(X), y_f32)[0], n_row)
    return _new(stream, n, _U8_TYPE, X.device, out=False) if n else None


def gemm_grouped(fmt: int, W, rows: int, in_dim: int, X, offsets, order=None, per: int = 1, Y=None, *,
                 act: int = ACT_NONE, up=None, bias=None, up_bias=None, alpha: float = 1.702, limit: float = 7.0,
                 residual=None, workspace=None, stream=None, y_f32: bool = False):
    """rf_gemm_grouped: row r of Y, in group g (offsets[g] <= r < offsets[g +
    1]), is residual + act(W_g x + bias_g, up_g x + up_bias_g), where x is row
    r of X, or row order[r] // per.  W and up are (n_group, rows, in_dim)
    quantized, offsets (n_group + 1,) and order (n_row,) int32 device tensors,
    biases (n_group, rows) float32.  Y and residual are of X's type, with y_f32
    float32.  Rows of no group are left as they were (a Y made here holds
    anything there)."""
    _known_fmt(fmt)
    px, ldx, n_x, n, dt = _matrix_rows(X, "X")
    if n != in_dim:
        raise ValueError(f"X must be (n, {in_dim})")
    for t, what in ((offsets, "offsets"), (order, "order")):
        if t is not None and (not t.is_cuda or t.element_size() != 4 or t.is_floating_point() or t.dim() != 1 or
                              not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous int32 CUDA tensor")
    n_group, n_row = offsets.numel() - 1, n_x if order is None else order.numel()
    dt, dty = _product_types(dt, y_f32)
    if Y is None:
        Y = _new(stream, (n_row, rows), _F32_TYPE if y_f32 else X.dtype, X.device)
    py, ldy = _rows(Y, n_row, rows, dty, "Y")
    e = _epilogue(max(n_group, 0) * rows, n_row, rows, dty, act, up, bias, up_bias, alpha, limit, residual)
    if workspace is None:
        need = lib().rf_gemm_grouped_workspace_bytes(fmt, n_group, rows, in_dim, dt, n_row)
    workspace, ws, ws_bytes = _space(workspace, need if workspace is None else 0, stream, X.device)
    _check(lib().rf_gemm_grouped(fmt, _weights(W, max(n_group, 0) * rows, fmt, in_dim, "W"),
                                 None if up is None else _weights(up, max(n_group, 0) * rows, fmt, in_dim, "up"),
                                 n_group, rows, in_dim, dt, px, ldx, n_x, offsets.data_ptr(),
                                 None if order is None else order.data_ptr(), per, n_row, ctypes.byref(e), py, ldy, ws,
                                 ws_bytes, _stream(stream)), "rf_gemm_grouped")
    return Y


class MoERouting:
    """What rf_moe_route_tokens gives: idx (int32) and w (float32), (n_tok,
    top_k); offsets (n_expert + 1,), order and place (n_tok * top_k,), int32."""

    def __init__(self, n_tok: int, n_expert: int, top_k: int, device, stream=None):
        if _empty is None:
            _look_up()
        n = n_tok * top_k
        self.idx = _new(stream, (n_tok, top_k), _I32_TYPE, device)
        self.w = _new(stream, (n_tok, top_k), _F32_TYPE, device)
        self.offsets = _new(stream, n_expert + 1, _I32_TYPE, device)
        self.order = _new(stream, n, _I32_TYPE, device)
        self.place = _new(stream, n, _I32_TYPE, device)


def moe_route_tokens(logits, top_k: int, workspace=None, stream=None) -> MoERouting:
    """rf_moe_route_tokens: logits (n_tok, n_expert) float32, float16 or
    bfloat16 (rows may be strided)."""
    pl, ld, n_tok, n_expert, dt = _matrix_rows(logits, "logits")
    r = MoERouting(n_tok, n_expert, max(top_k, 0), logits.device, stream)
    if workspace is None:
        need = lib().rf_moe_route_tokens_workspace_bytes(n_tok, n_expert, top_k)
    workspace, ws, ws_bytes = _space(workspace, need if workspace is None else 0, stream, logits.device)
    _check(lib().rf_moe_route_tokens(dt, pl, ld, n_tok, n_expert, top_k, r.idx.data_ptr(), r.w.data_ptr(),
                                     r.offsets.data_ptr(), r.order.data_ptr(), r.place.data_ptr(), ws, ws_bytes,
                                     _stream(stream)), "rf_moe_route_tokens")
    return r


def moe_tokens_workspace(fmt: int, n_expert: int, top_k: int, n_ff: int, n_embd: int, X, stream=None):
    """Device workspace for moe_ffn_tokens() of X on `stream`, or None."""
    n = lib().rf_moe_tokens_workspace_bytes(fmt, n_expert, top_k, n_ff, n_embd, _dtype(X), X.shape[0])
    return _new(stream, n, _U8_TYPE, X.device, out=False) if n else None


def moe_ffn_tokens(fmt: int, logits, top_k: int, gate, up, down, n_ff: int, n_embd: int, X, Y=None, *, gate_bias=None,
                   up_bias=None, down_bias=None, alpha: float | None = None, limit: float | None = None, residual=None,
                   workspace=None, stream=None):
    """rf_moe_ffn_tokens: the routed FFN of a chunk X (n_tok, n_embd) over
    stacked experts, with the clamped SwiGLU when alpha and limit are given and
    the plain one without.  logits (n_tok, n_expert) may be of another type
    than X; biases are float32.  Returns Y (n_tok, n_embd), of X's type."""
    _known_fmt(fmt)
    px, ldx, n_tok, n, dt = _matrix_rows(X, "X")
    pl, ldl, nl, n_expert, ldt = _matrix_rows(logits, "logits")
    if n != n_embd or nl != n_tok:
        raise ValueError(f"X must be (n_tok, {n_embd}), logits (n_tok, n_expert)")
    if (alpha is None) != (limit is None):
        raise ValueError("alpha and limit belong together")
    if Y is None:
        Y = _new(stream, (n_tok, n_embd), X.dtype, X.device)
    py, ldy = _rows(Y, n_tok, n_embd, dt, "Y")
    pr, ldr = _rows(residual, n_tok, n_embd, dt, "residual")
    if workspace is None:
        need = lib().rf_moe_tokens_workspace_bytes(fmt, n_expert, top_k, n_ff, n_embd, dt, n_tok)
    workspace, ws, ws_bytes = _space(workspace, need if workspace is None else 0, stream, X.device)
    clamped = alpha is not None
    _check(lib().rf_moe_ffn_tokens(fmt, dt, ldt, pl, ldl, n_expert, top_k, n_tok,
                                   _weights(gate, n_expert * n_ff, fmt, n_embd, "gate"),
                                   _weights(up, n_expert * n_ff, fmt, n_embd, "up"),
                                   _weights(down, n_expert * n_embd, fmt, n_ff, "down"),
                                   _f32_ptr(gate_bias, n_expert * n_ff, "gate_bias"),
                                   _f32_ptr(up_bias, n_expert * n_ff, "up_bias"),
                                   _f32_ptr(down_bias, n_expert * n_embd, "down_bias"),
                                   ACT_SWIGLU_CLAMPED if clamped else ACT_SWIGLU, alpha if clamped else 0.0,
                                   limit if clamped else 0.0, n_ff, n_embd, px, ldx, pr, ldr, py, ldy, ws, ws_bytes,
                                   _stream(stream)), "rf_moe_ffn_tokens")
    return Y


def device_status() -> int:
    """Synchronize and return (and clear) the kernels' device status word."""
    return lib().rf_device_status()


def debug_arm_wait_fault(limit_us: int) -> None:
    """rf_debug_arm_wait_fault (test hook): the next tensor-copy GEMV launch
    withholds one stage's copy and gives up its wait after limit_us."""
    _check(lib().rf_debug_arm_wait_fault(limit_us), "rf_debug_arm_wait_fault")


def debug_attention_plan(cache: KVCache, batch: KVBatch, q, window: int = 0, max_len: int = 0) -> dict:
    """rf_debug_attention_plan (test hook): how attention() lays out a call
    with these arguments."""
    p = AttentionPlan()
    _check(lib().rf_debug_attention_plan(cache.ref, batch.ref, _dtype(q), q.shape[1], window, max_len,
                                         ctypes.byref(p)), "rf_debug_attention_plan")
    return {k: getattr(p, k) for k, _ in AttentionPlan._fields_ if k != "reserved"}
