"""Python binding of libloco.so (ctypes): argument marshalling only.

Every function takes torch tensors (device memory) and passes their pointers, sizes and
the current HIP stream to the C ABI of the same name; every step of the computation
runs in the library's HIP kernels.  There is no fallback: if the library is missing or
a call returns an error status, the call raises.
"""

from __future__ import annotations

import ctypes
import math
import operator
import os
import warnings

import torch

from . import build as _build

LOCO_F32 = 0
LOCO_BF16 = 1
LOCO_I8 = 2
LOCO_OK = 0
LOCO_ERR_INVALID = -1
LOCO_ERR_ALIGN = -2
LOCO_ERR_UNSUPPORTED = -3
LOCO_ERR_HIP = -4
LOCO_MAX_PEERS = 128
LOCO_ACT_NONE = 0
LOCO_ACT_RELU = 1
LOCO_ACT_GELU = 2
LOCO_ACT_SILU = 3
LOCO_GATE_NONE = 0
LOCO_GATE_COLUMN = 1
LOCO_GATE_ELEMENT = 2
LOCO_MAX_TOP = 32

SYMBOLS = ["loco_compensate_quantize", "loco_compensate_quantize_ex", "loco_dequant_reduce",
           "loco_dequant_reduce_adam", "loco_topk_quantize", "loco_sparse_aggregate", "loco_status_string",
           "loco_version", "loco_layer_norm", "loco_layer_norm_backward", "loco_layer_norm_backward_workspace",
           "loco_checkpoint_write", "loco_checkpoint_read", "loco_linear", "loco_linear_workspace",
           "loco_linear_input_grad", "loco_linear_input_grad_workspace", "loco_linear_weight_grad",
           "loco_linear_weight_grad_workspace", "loco_adamw_table_bytes", "loco_adamw_plan",
           "loco_adamw", "loco_adamw_ex", "loco_adamw_state_plan", "loco_adamw_state_read", "loco_adamw_state_write",
           "loco_residual_norm", "loco_residual_norm_backward", "loco_residual_norm_backward_workspace",
           "loco_token_logprobs", "loco_token_logprobs_workspace", "loco_token_logprobs_backward",
           "loco_token_logprobs_ex", "loco_token_logprobs_backward_ex"]


class LocoError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} ({status})")


class CqSegment(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("err", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("absmax", ctypes.c_void_p), ("n", ctypes.c_int64)]


class CqOptions(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("block", ctypes.c_int), ("beta", ctypes.c_float),
                ("fixed_scale", ctypes.c_float), ("err_scale", ctypes.c_float),
                ("reset_error", ctypes.c_int)]


class Payload(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p)]


class AdamParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("delta", ctypes.c_float)]


class SparsePayload(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p)]


class Checkpoint(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p), ("block", ctypes.c_int)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_exps", ctypes.c_void_p), ("v_exps", ctypes.c_void_p), ("param_bf16", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("weight_decay", ctypes.c_double)]


class AdamwOptions(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64)]


class AdamwRounding(ctypes.Structure):
    _fields_ = [("seed", ctypes.c_uint64), ("counter", ctypes.c_void_p)]


class AdamwState(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p), ("values", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("moment", ctypes.c_int)]


class AdamwPlan(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("ntensors", ctypes.c_int), ("live", ctypes.c_int64), ("tiles", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("tensors", ctypes.POINTER(AdamwTensor)), ("param_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("state_bits", ctypes.c_int), ("block", ctypes.c_int)]


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load libloco.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"HIP library not built: {path} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    lib.loco_compensate_quantize.argtypes = [ctypes.POINTER(CqSegment), ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                             ctypes.c_float, ctypes.c_void_p]
    lib.loco_compensate_quantize.restype = ctypes.c_int
    lib.loco_compensate_quantize_ex.argtypes = [ctypes.POINTER(CqSegment), ctypes.c_int, ctypes.c_int,
                                                ctypes.c_int, ctypes.POINTER(CqOptions), ctypes.c_void_p]
    lib.loco_compensate_quantize_ex.restype = ctypes.c_int
    lib.loco_dequant_reduce.argtypes = [ctypes.POINTER(Payload), ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                        ctypes.c_int, ctypes.c_void_p]
    lib.loco_dequant_reduce.restype = ctypes.c_int
    lib.loco_dequant_reduce_adam.argtypes = [ctypes.POINTER(Payload), ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_float, ctypes.c_float, ctypes.POINTER(AdamParams),
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p]
    lib.loco_dequant_reduce_adam.restype = ctypes.c_int
    lib.loco_topk_quantize.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                       ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    lib.loco_topk_quantize.restype = ctypes.c_int
    lib.loco_sparse_aggregate.argtypes = [ctypes.POINTER(SparsePayload), ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_void_p]
    lib.loco_sparse_aggregate.restype = ctypes.c_int
    ptr, i32, i64, f32, ckpt = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.POINTER(Checkpoint))
    for fn, res, args in (
            ("loco_layer_norm", i32, [ptr, i32, ptr, ptr, i32, i64, i64, f32, ptr, ptr, ptr, ckpt, ptr]),
            ("loco_layer_norm_backward", i32, [ptr, ptr, i32, ptr, i32, ptr, ptr, ptr, i64, i64, ptr, ptr, ptr, i32,
                                               ptr, i64, ptr]),
            ("loco_layer_norm_backward_workspace", i64, [i64, i64]),
            ("loco_checkpoint_write", i32, [ptr, i32, i64, i64, ckpt, ptr]),
            ("loco_checkpoint_read", i32, [ckpt, i64, i64, i32, ptr, i32, ptr]),
            ("loco_linear", i32, [ptr, ptr, ptr, ptr, i64, i64, i64, i32, ptr, i32, ckpt, ptr, i64, ptr]),
            ("loco_linear_workspace", i64, [i64, i64, i64]),
            ("loco_linear_input_grad", i32, [ptr, ptr, ptr, i64, i64, i64, i32, ckpt, ptr, i32, ptr, i64, ptr]),
            ("loco_linear_input_grad_workspace", i64, [i64, i64, i64]),
            ("loco_linear_weight_grad", i32, [ptr, ckpt, i64, i64, i64, i32, i32, ptr, ptr, i32, ptr, i64, ptr]),
            ("loco_linear_weight_grad_workspace", i64, [i64, i64, i64, i32]),
            ("loco_residual_norm", i32, [ptr, ptr, i32, ptr, i32, ptr, ptr, i32, i64, i64, f32, f32, ptr, ptr, ptr, ptr,
                                         ckpt, ptr]),
            ("loco_residual_norm_backward", i32, [ptr, ptr, ptr, ptr, i32, ptr, i32, ptr, ptr, i32, ptr, ptr, i64, i64,
                                                  f32, ptr, ptr, ptr, ptr, ptr, i32, ptr, i64, ptr]),
            ("loco_residual_norm_backward_workspace", i64, [i64, i64]),
            ("loco_token_logprobs", i32, [ptr, i32, i64, i64, i64, ptr, f32, ptr, ptr, ptr, i32, ptr, ptr, ptr, i64, ptr]),
            ("loco_token_logprobs_ex", i32, [ptr, i32, i64, i64, i64, i64, i64, ptr, i64, f32, ptr, ptr, ptr, i32, ptr, ptr,
                                             ptr, i64, ptr]),
            ("loco_token_logprobs_workspace", i64, [i64, i64, i32]),
            ("loco_token_logprobs_backward_ex", i32, [ptr, i32, i64, i64, i64, i64, i64, ptr, i64, f32, ptr, ptr, ptr, ptr,
                                                      ptr, i64, i64, ptr]),
            ("loco_token_logprobs_backward", i32, [ptr, i32, i64, i64, i64, ptr, f32, ptr, ptr, ptr, ptr, ptr, i64, ptr]),
            ("loco_adamw_table_bytes", i64, [i32]),
            ("loco_adamw_plan", i32, [ctypes.POINTER(AdamwTensor), i32, i32, i32, i32, i32, ptr, i64,
                                      ctypes.POINTER(AdamwPlan), ptr]),
            ("loco_adamw", i32, [ctypes.POINTER(AdamwPlan), ctypes.POINTER(AdamwOptions), ptr, ptr]),
            ("loco_adamw_ex", i32, [ctypes.POINTER(AdamwPlan), ctypes.POINTER(AdamwOptions), ptr,
                                    ctypes.POINTER(AdamwRounding), ptr]),
            ("loco_adamw_state_plan", i32, [ctypes.POINTER(AdamwState), i32, i32, i32, ptr, i64,
                                            ctypes.POINTER(AdamwPlan), ptr]),
            ("loco_adamw_state_read", i32, [ctypes.POINTER(AdamwPlan), ptr]),
            ("loco_adamw_state_write", i32, [ctypes.POINTER(AdamwPlan), ptr])):
        getattr(lib, fn).argtypes = args
        getattr(lib, fn).restype = res
    lib.loco_status_string.argtypes = [ctypes.c_int]
    lib.loco_status_string.restype = ctypes.c_char_p
    lib.loco_version.argtypes = []
    lib.loco_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().loco_status_string(int(status)).decode()


loco_status_string = status_string


def _check(fn, status):
    if status != LOCO_OK:
        raise LocoError(fn, status)


def _dtype_code(t: torch.Tensor) -> int:
    if t is None:  # a missing buffer: the C call refuses its null pointer
        return LOCO_F32
    if t.dtype == torch.float32:
        return LOCO_F32
    if t.dtype == torch.bfloat16:
        return LOCO_BF16
    if t.dtype == torch.int8:
        return LOCO_I8
    raise TypeError(f"unsupported dtype {t.dtype}")


try:  # the current stream's handle without building a Stream object (~2.5 us less per call)
    _current_raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # pragma: no cover - a torch without it
    _current_raw_stream = None


def _device() -> int:
    """The current device: every call launches there, so its tensors must live there."""
    return torch.cuda.current_device()


def _ptr(t, dev):
    if t is None:
        return None
    d = t.get_device()
    if d != dev:
        if d < 0:
            raise ValueError("tensor must be in device memory")
        raise ValueError(f"tensor is on cuda:{d}; the call runs on the current device, cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream, dev):
    if stream is None:
        if _current_raw_stream is not None:
            return _current_raw_stream(dev)
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def code_bytes(n: int, bits: int) -> int:
    return (n * bits + 7) // 8


def num_blocks(n: int, block: int) -> int:
    return -(-n // block)


# Sizes the C calls accept; for these, the binding checks that every tensor holds the bytes
# the call will read or write (the C ABI sees only pointers and n).  Other values go to
# the C call unchecked, which refuses them with its own status.
_BITS = (2, 4, 8)
_BLOCKS = (64, 128, 256, 512)
_CHUNKS = (256, 512, 1024, 2048, 4096)


def _need(t, nbytes: int, what: str) -> None:
    if t is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{what} holds {t.numel() * t.element_size()} bytes; the call needs {nbytes}")


def _segments(segments, dev, bits=None, block=None, fixed=False):
    segs = list(segments)
    arr = (CqSegment * max(1, len(segs)))()
    gd = ed = None
    for i, (g, e, c, a) in enumerate(segs):
        gi, ei = _dtype_code(g), _dtype_code(e)
        gd = gi if gd is None else gd
        ed = ei if ed is None else ed
        if gi != gd or ei != ed:
            raise TypeError("all segments must share grad and err dtypes")
        n = g.numel()
        if e.numel() != n:
            raise ValueError(f"segment {i}: err has {e.numel()} elements, grad {n}")
        if n > 0 and bits in _BITS:
            _need(c, code_bytes(n, bits), f"segment {i}: codes")
            if not fixed and block in _BLOCKS:
                _need(a, 4 * num_blocks(n, block), f"segment {i}: absmax")
        arr[i] = CqSegment(_ptr(g, dev), _ptr(e, dev), _ptr(c, dev), _ptr(a, dev), n)
    return arr, len(segs), gd, ed


def _payloads(peers, dev, n, bits, block, fixed):
    ps = list(peers)
    arr = (Payload * max(1, len(ps)))()
    for i, (c, a) in enumerate(ps):
        if n > 0 and bits in _BITS:
            _need(c, code_bytes(n, bits), f"peer {i}: codes")
            if not fixed and block in _BLOCKS:
                _need(a, 4 * num_blocks(n, block), f"peer {i}: absmax")
        arr[i] = Payload(_ptr(c, dev), _ptr(a, dev))
    return arr, ps


def loco_compensate_quantize(segments, *, bits: int, block: int, beta: float, fixed_scale: float = 0.0,
                             stream=None, grad_dtype=None, err_dtype=None) -> None:
    """segments: iterable of (grad, err, codes, absmax) tensors; absmax may be None in
    fixed-scale mode.  n of a segment is grad.numel()."""
    dev = _device()
    arr, nseg, gd, ed = _segments(segments, dev, bits, block, fixed_scale > 0)
    gd = gd if grad_dtype is None else grad_dtype
    ed = ed if err_dtype is None else err_dtype
    st = load().loco_compensate_quantize(arr, nseg, LOCO_F32 if gd is None else gd,
                                         LOCO_F32 if ed is None else ed, bits, block, beta,
                                         fixed_scale, _stream(stream, dev))
    _check("loco_compensate_quantize", st)


def loco_compensate_quantize_ex(segments, *, bits: int, block: int, beta: float, fixed_scale: float = 0.0,
                                err_scale: float = 0.0, reset_error: bool = False, stream=None,
                                grad_dtype=None, err_dtype=None) -> None:
    """As loco_compensate_quantize; an int8 err tensor holds the 8-bit error of scale
    err_scale, and reset_error stores a zero error this step."""
    dev = _device()
    arr, nseg, gd, ed = _segments(segments, dev, bits, block, fixed_scale > 0)
    gd = gd if grad_dtype is None else grad_dtype
    ed = ed if err_dtype is None else err_dtype
    opt = CqOptions(bits, block, beta, fixed_scale, err_scale, 1 if reset_error else 0)
    st = load().loco_compensate_quantize_ex(arr, nseg, LOCO_F32 if gd is None else gd,
                                            LOCO_F32 if ed is None else ed, ctypes.byref(opt),
                                            _stream(stream, dev))
    _check("loco_compensate_quantize_ex", st)


def loco_dequant_reduce(peers, n: int, *, bits: int, block: int, out, out_scale: float,
                        fixed_scale: float = 0.0, stream=None) -> None:
    """peers: iterable of (codes, absmax) tensors (absmax None in fixed-scale mode)."""
    dev = _device()
    arr, ps = _payloads(peers, dev, n, bits, block, fixed_scale > 0)
    if out is not None:
        _need(out, n * out.element_size(), "out")
    st = load().loco_dequant_reduce(arr if ps else None, len(ps), n, bits, block, fixed_scale, out_scale,
                                    _ptr(out, dev), _dtype_code(out), _stream(stream, dev))
    _check("loco_dequant_reduce", st)


def loco_dequant_reduce_adam(peers, n: int, *, bits: int, block: int, out_scale: float, param, m, v,
                             lr: float, beta1: float, beta2: float, delta: float, param_bf16=None,
                             fixed_scale: float = 0.0, stream=None) -> None:
    """peers as loco_dequant_reduce; param, m, v float32 tensors of n elements, updated in
    place; param_bf16 an optional bfloat16 tensor that receives the new param."""
    for t in (param, m, v):
        if t.dtype != torch.float32:
            raise TypeError("param, m and v must be float32")
    if param_bf16 is not None and param_bf16.dtype != torch.bfloat16:
        raise TypeError("param_bf16 must be bfloat16")
    dev = _device()
    arr, ps = _payloads(peers, dev, n, bits, block, fixed_scale > 0)
    for t, what in ((param, "param"), (m, "m"), (v, "v")):
        _need(t, 4 * n, what)
    _need(param_bf16, 2 * n, "param_bf16")
    hp = AdamParams(lr, beta1, beta2, delta)
    st = load().loco_dequant_reduce_adam(arr if ps else None, len(ps), n, bits, block, fixed_scale, out_scale,
                                         ctypes.byref(hp), _ptr(param, dev), _ptr(m, dev), _ptr(v, dev),
                                         _ptr(param_bf16, dev), _stream(stream, dev))
    _check("loco_dequant_reduce_adam", st)


def loco_topk_quantize(grad, err, *, chunk: int, k: int, idx, codes, absmax, bits: int = 2,
                       ef_decay: float = 1.0, stream=None) -> None:
    if grad.dtype != torch.float32 or err.dtype != torch.float32:
        raise TypeError("grad and err must be float32")
    dev = _device()
    n = grad.numel()
    if err.numel() != n:
        raise ValueError(f"err has {err.numel()} elements, grad {n}")
    if n > 0 and chunk in _CHUNKS and 1 <= k <= chunk and bits in _BITS:
        chunks = num_blocks(n, chunk)
        _need(idx, 2 * chunks * k, "idx")
        _need(codes, chunks * code_bytes(k, bits), "codes")
        _need(absmax, 4 * chunks, "absmax")
    st = load().loco_topk_quantize(_ptr(grad, dev), _ptr(err, dev), grad.numel(), chunk, k, bits, ef_decay,
                                   _ptr(idx, dev), _ptr(codes, dev), _ptr(absmax, dev), _stream(stream, dev))
    _check("loco_topk_quantize", st)


def loco_sparse_aggregate(peers, n: int, *, chunk: int, k: int, out, out_scale: float, bits: int = 2,
                          stream=None) -> None:
    """peers: iterable of (idx int16/uint16, codes uint8, absmax float32) tensors, as
    loco_topk_quantize writes them."""
    dev = _device()
    ps = list(peers)
    arr = (SparsePayload * max(1, len(ps)))()
    check = n > 0 and chunk in _CHUNKS and 1 <= k <= chunk and bits in _BITS
    chunks = num_blocks(n, chunk) if check else 0
    for i, (ix, c, a) in enumerate(ps):
        if check:
            _need(ix, 2 * chunks * k, f"peer {i}: idx")
            _need(c, chunks * code_bytes(k, bits), f"peer {i}: codes")
            _need(a, 4 * chunks, f"peer {i}: absmax")
        arr[i] = SparsePayload(_ptr(ix, dev), _ptr(c, dev), _ptr(a, dev))
    if check and out is not None:
        _need(out, n * out.element_size(), "out")
    st = load().loco_sparse_aggregate(arr if ps else None, len(ps), n, chunk, k, bits, out_scale, _ptr(out, dev),
                                      _dtype_code(out), _stream(stream, dev))
    _check("loco_sparse_aggregate", st)


# -- layer operators ---------------------------------------------------------------------
#
# A matrix is a contiguous tensor whose last dimension is its columns; the leading ones
# together are its rows (tokens).  A checkpoint is a pair (codes int8, exps uint8), with
# the block (32 or 64) given beside it.  The call's first matrix sets the sizes; the others
# have its leading dimensions, or one for all rows, or are flat (one dimension for the whole).

# These calls are short beside a small kernel's launch, so the checks make few torch calls:
# sizes and types first, then (_ptr) where each tensor lies.

_F32 = (torch.float32,)
_BF = (torch.bfloat16,)
_FLOATS = (torch.float32, torch.bfloat16)
_CODES = {torch.float32: LOCO_F32, torch.bfloat16: LOCO_BF16}


def _rows_cols(t, what, dtypes):
    shape = t.shape
    if not shape:
        raise ValueError(f"{what} must have at least one dimension")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if len(shape) == 2:
        return shape
    cols = shape[-1]
    return (t.numel() // cols if cols else math.prod(shape[:-1])), cols


def _sized(t, numel: int, what: str, dtypes) -> None:
    """t (None passes: the C call decides) must hold exactly numel elements of one of dtypes."""
    if t is None:
        return
    if t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements; the call needs {numel}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")


def _matrix(t, like, rows, cols, what: str, dtypes) -> None:
    """As _sized, for a matrix whose rows are those of the shape `like`: one with as many elements
    but laid out otherwise would be filled as another matrix."""
    if t is None:
        return
    shape = t.shape
    if shape != (rows, cols):
        _sized(t, rows * cols, what, dtypes)
        lead, shape = tuple(like)[:-1], tuple(shape)
        if len(shape) > 1 and not (shape[-1] == cols and _same_rows(shape[:-1], lead)):
            raise ValueError(f"{what} has the shape {shape}; the call's is {(*lead, cols)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")


def _per_row(t, like, rows, what: str) -> None:
    """As _sized, for one float32 per row of the shape `like`."""
    _sized(t, rows, what, _F32)
    if t is not None and t.dim() > 1 and not _same_rows(tuple(t.shape), tuple(like)[:-1]):
        raise ValueError(f"{what} has the shape {tuple(t.shape)}; the call's is {tuple(like)[:-1]}")


def _same_rows(a, b) -> bool:
    """Whether leading dimensions a and b, of as many rows, count them in the same order."""
    if a == b or len(a) <= 1 or len(b) <= 1:
        return True
    a, b = [d for d in a if d != 1], [d for d in b if d != 1]
    return a == b or len(a) <= 1 or len(b) <= 1


def _checkpoint(checkpoint, block, like, rows, cols, dev):
    """The C struct of (codes, exps), or None."""
    if checkpoint is None:
        return None
    codes, exps = checkpoint
    _matrix(codes, like, rows, cols, "checkpoint codes", (torch.int8,))
    if block in (32, 64):
        _matrix(exps, like, rows, num_blocks(cols, block), "checkpoint exps", (torch.uint8,))
    return ctypes.byref(Checkpoint(_ptr(codes, dev), _ptr(exps, dev), block))


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def loco_layer_norm(x, weight, bias, *, out, mean, rstd, eps: float = 1e-5, checkpoint=None, block: int = 64,
                    stream=None) -> None:
    """out = (x - mean) * rstd * weight + bias over x's last dimension; mean and rstd
    (float32, one per row) are written for the backward pass, and `checkpoint`, if given,
    with the 8-bit checkpoint of the output.  weight and bias may be None."""
    dev = _device()
    rows, cols = _rows_cols(x, "x", _FLOATS)
    like = x.shape
    _matrix(out, like, rows, cols, "out", (x.dtype,))
    param = weight if weight is not None else bias
    _sized(weight, cols, "weight", _FLOATS)
    _sized(bias, cols, "bias", _FLOATS if weight is None else (weight.dtype,))
    _per_row(mean, like, rows, "mean")
    _per_row(rstd, like, rows, "rstd")
    ck = _checkpoint(checkpoint, block, like, rows, cols, dev)
    st = (_lib or load()).loco_layer_norm(
        _ptr(x, dev), _CODES[x.dtype], _ptr(weight, dev), _ptr(bias, dev),
        LOCO_F32 if param is None else _CODES[param.dtype], rows, cols, eps, _ptr(out, dev), _ptr(mean, dev),
        _ptr(rstd, dev), ck, _stream(stream, dev))
    _check("loco_layer_norm", st)


def loco_layer_norm_backward(dy, x, weight, mean, rstd, *, dx, dweight=None, dbias=None, residual=None,
                             workspace=None, stream=None) -> None:
    """dx of loco_layer_norm (plus residual, if given), and dweight and dbias summed over the
    rows, each optional.  workspace: a tensor of layer_norm_backward_workspace(rows, cols)
    bytes, not needed without dweight and dbias."""
    dev = _device()
    rows, cols = _rows_cols(x, "x", _FLOATS)
    like = x.shape
    for t, what in ((dy, "dy"), (dx, "dx"), (residual, "residual")):
        _matrix(t, like, rows, cols, what, (x.dtype,))
    _sized(weight, cols, "weight", _FLOATS)
    _per_row(mean, like, rows, "mean")
    _per_row(rstd, like, rows, "rstd")
    grad = dweight if dweight is not None else dbias
    _sized(dweight, cols, "dweight", _FLOATS)
    _sized(dbias, cols, "dbias", _FLOATS if dweight is None else (dweight.dtype,))
    st = (_lib or load()).loco_layer_norm_backward(
        _ptr(dy, dev), _ptr(x, dev), _CODES[x.dtype], _ptr(weight, dev),
        LOCO_F32 if weight is None else _CODES[weight.dtype], _ptr(mean, dev), _ptr(rstd, dev), _ptr(residual, dev),
        rows, cols, _ptr(dx, dev), _ptr(dweight, dev), _ptr(dbias, dev),
        LOCO_F32 if grad is None else _CODES[grad.dtype], _ptr(workspace, dev), _nbytes(workspace),
        _stream(stream, dev))
    _check("loco_layer_norm_backward", st)


def loco_layer_norm_backward_workspace(rows: int, cols: int) -> int:
    return load().loco_layer_norm_backward_workspace(rows, cols)


def loco_checkpoint_write(x, *, codes, exps, block: int = 64, stream=None) -> None:
    """The 8-bit checkpoint of x: codes int8 of x's shape, exps uint8, one per block of a row."""
    dev = _device()
    rows, cols = _rows_cols(x, "x", _FLOATS)
    ck = _checkpoint((codes, exps), block, x.shape, rows, cols, dev)
    st = (_lib or load()).loco_checkpoint_write(
        _ptr(x, dev), _CODES[x.dtype], rows, cols, ck, _stream(stream, dev))
    _check("loco_checkpoint_write", st)


def loco_checkpoint_read(codes, exps, *, out, block: int = 64, act: int = LOCO_ACT_NONE, stream=None) -> None:
    """out = act(the values of the checkpoint); the matrix's shape is out's."""
    dev = _device()
    rows, cols = _rows_cols(out, "out", _FLOATS)
    ck = _checkpoint((codes, exps), block, out.shape, rows, cols, dev)
    st = (_lib or load()).loco_checkpoint_read(
        ck, rows, cols, act, _ptr(out, dev), _CODES[out.dtype], _stream(stream, dev))
    _check("loco_checkpoint_read", st)


def loco_linear(x, weight, *, out, bias=None, act: int = LOCO_ACT_NONE, residual=None, checkpoint=None,
                block: int = 64, workspace=None, stream=None) -> None:
    """out = act(x weight^T + bias) + residual, with weight [out_features, in_features];
    `checkpoint`, if given, is written with the 8-bit checkpoint of the activation's input.
    bfloat16, out bfloat16 or float32.  workspace: a tensor of linear_workspace(rows,
    out_features, in_features) bytes; up to 16 rows of at most 4096 features need none without
    a checkpoint."""
    dev = _device()
    rows, k = _rows_cols(x, "x", _BF)
    n, wk = _rows_cols(weight, "weight", _BF)
    if wk != k:
        raise ValueError(f"x has {k} columns, weight {wk}")
    _sized(bias, n, "bias", _BF)
    like = x.shape
    _matrix(residual, like, rows, n, "residual", _BF)
    _matrix(out, like, rows, n, "out", _FLOATS)
    ck = _checkpoint(checkpoint, block, like, rows, n, dev)
    st = (_lib or load()).loco_linear(
        _ptr(x, dev), _ptr(weight, dev), _ptr(bias, dev), _ptr(residual, dev), rows, n, k, act, _ptr(out, dev),
        _CODES[out.dtype], ck, _ptr(workspace, dev), _nbytes(workspace), _stream(stream, dev))
    _check("loco_linear", st)


def loco_linear_workspace(rows: int, out_features: int, in_features: int) -> int:
    return load().loco_linear_workspace(rows, out_features, in_features)


def loco_linear_input_grad(dy, weight, *, out, act: int = LOCO_ACT_NONE, checkpoint=None, block: int = 64,
                           residual=None, workspace=None, stream=None) -> None:
    """out = (dy weight) * act'(z) + residual, with z read from the 8-bit checkpoint of the
    activation's input (needed unless act is LOCO_ACT_NONE)."""
    dev = _device()
    rows, n = _rows_cols(dy, "dy", _BF)
    wn, k = _rows_cols(weight, "weight", _BF)
    if wn != n:
        raise ValueError(f"dy has {n} columns, weight {wn} rows")
    like = dy.shape
    _matrix(residual, like, rows, k, "residual", _BF)
    _matrix(out, like, rows, k, "out", _FLOATS)
    ck = _checkpoint(checkpoint, block, like, rows, k, dev)
    st = (_lib or load()).loco_linear_input_grad(
        _ptr(dy, dev), _ptr(weight, dev), _ptr(residual, dev), rows, n, k, act, ck, _ptr(out, dev), _CODES[out.dtype],
        _ptr(workspace, dev), _nbytes(workspace), _stream(stream, dev))
    _check("loco_linear_input_grad", st)


def loco_linear_input_grad_workspace(rows: int, out_features: int, in_features: int) -> int:
    return load().loco_linear_input_grad_workspace(rows, out_features, in_features)


def loco_linear_weight_grad(dy, checkpoint, *, out, block: int = 64, act: int = LOCO_ACT_NONE, dbias=None,
                            accumulate: bool = False, workspace=None, stream=None) -> None:
    """out [out_features, in_features] = dy^T act(the checkpoint's values), dbias = dy summed
    over the rows; with accumulate, added to what they hold.  out and dbias are bfloat16
    or float32, alike.  GELU's and SiLU's values are rounded to bfloat16 for bfloat16 gradients
    and enter as two bfloat16 numbers, in twice the time, for float32 ones."""
    dev = _device()
    rows, n = _rows_cols(dy, "dy", _BF)
    wn, k = _rows_cols(out, "out", _FLOATS)
    if wn != n:
        raise ValueError(f"dy has {n} columns, out {wn} rows")
    _sized(dbias, n, "dbias", (out.dtype,))
    ck = _checkpoint(checkpoint, block, dy.shape, rows, k, dev)
    st = (_lib or load()).loco_linear_weight_grad(
        _ptr(dy, dev), ck, rows, n, k, act, 1 if accumulate else 0, _ptr(out, dev), _ptr(dbias, dev),
        _CODES[out.dtype], _ptr(workspace, dev), _nbytes(workspace), _stream(stream, dev))
    _check("loco_linear_weight_grad", st)


def loco_linear_weight_grad_workspace(rows: int, out_features: int, in_features: int,
                                      act: int = LOCO_ACT_NONE) -> int:
    return load().loco_linear_weight_grad_workspace(rows, out_features, in_features, act)


# -- the norms around a block -----------------------------------------------------------------

def _params(cols, *named) -> int:
    """The type code of the parameters given (all alike), each of cols elements."""
    dtype = None
    for t, what in named:
        if t is None:
            continue
        _sized(t, cols, what, _FLOATS if dtype is None else (dtype,))
        dtype = t.dtype
    return LOCO_F32 if dtype is None else _CODES[dtype]


def _gate(gate, like, rows, cols, dtype) -> int:
    """LOCO_GATE_COLUMN for one dimension of cols elements, else LOCO_GATE_ELEMENT."""
    if gate is None:
        return LOCO_GATE_NONE
    if gate.dim() == 1 and gate.shape[0] == cols:
        return LOCO_GATE_COLUMN
    _matrix(gate, like, rows, cols, "gate", (dtype,))
    return LOCO_GATE_ELEMENT


def loco_residual_norm(y, residual, *, out=None, rstd=None, h=None, weight=None, post_rstd=None, post_weight=None,
                       gate=None, scale: float = 1.0, eps: float = 1e-5, checkpoint=None, block: int = 64,
                       stream=None) -> None:
    """What lies between two blocks, over the last dimension: u is y's RMS norm times post_weight if
    post_rstd (float32, one per row, written) is given, else y; h = residual + scale * gate * u; out =
    the RMS norm of h times weight, with rstd (float32, one per row) written for the backward pass, and
    `checkpoint`, if given, with the 8-bit checkpoint of out.  y may be None: the norm of the residual
    alone; so may residual.  gate has one dimension (a factor per column, of the weights' type) or the
    shape of y.  Without h the stream is not stored, without out (and rstd) it is not normed.
    post_weight goes with post_rstd."""
    dev = _device()
    x = residual if y is None else y
    if x is None:
        raise ValueError("y or residual is needed")
    rows, cols = _rows_cols(x, "residual" if y is None else "y", _FLOATS)
    like, dt = x.shape, (x.dtype,)
    for t, what in ((residual, "residual"), (h, "h"), (out, "out")):
        _matrix(t, like, rows, cols, what, dt)
    _per_row(rstd, like, rows, "rstd")
    _per_row(post_rstd, like, rows, "post_rstd")
    kind = _gate(gate, like, rows, cols, x.dtype)
    param = _params(cols, (weight, "weight"), (post_weight, "post_weight"),
                    (gate if kind == LOCO_GATE_COLUMN else None, "gate"))
    ck = _checkpoint(checkpoint, block, like, rows, cols, dev)
    st = (_lib or load()).loco_residual_norm(
        _ptr(y, dev), _ptr(residual, dev), _CODES[x.dtype], _ptr(gate, dev), kind, _ptr(post_weight, dev),
        _ptr(weight, dev), param, rows, cols, scale, eps, _ptr(h, dev), _ptr(out, dev), _ptr(post_rstd, dev),
        _ptr(rstd, dev), ck, _stream(stream, dev))
    _check("loco_residual_norm", st)


def loco_residual_norm_backward(dout, h=None, *, rstd=None, weight=None, dh=None, y=None, post_rstd=None,
                                post_weight=None, gate=None, scale: float = 1.0, dresidual=None, dy=None, dgate=None,
                                dweight=None, dpost_weight=None, workspace=None, stream=None) -> None:
    """The gradients of loco_residual_norm from those of out (dout) and of h (dh), either of which may be
    None, and what the forward pass left: h as stored (the norm's input), rstd, y, post_rstd.
    dresidual, dy and a gate of elements' dgate have their matrix's shape and type; dweight,
    dpost_weight and a gate of columns' dgate are summed over the rows, float32 or bfloat16,
    alike.  Each is optional.  workspace: a tensor of residual_norm_backward_workspace(rows, cols)
    bytes, not needed without sums over the rows."""
    dev = _device()
    x = dh if dout is None else dout
    if x is None:
        raise ValueError("dout or dh is needed")
    rows, cols = _rows_cols(x, "dh" if dout is None else "dout", _FLOATS)
    like, dt = x.shape, (x.dtype,)
    for t, what in ((dh, "dh"), (h, "h"), (y, "y"), (dresidual, "dresidual"), (dy, "dy")):
        _matrix(t, like, rows, cols, what, dt)
    _per_row(rstd, like, rows, "rstd")
    _per_row(post_rstd, like, rows, "post_rstd")
    kind = _gate(gate, like, rows, cols, x.dtype)
    columns = kind == LOCO_GATE_COLUMN
    if dgate is not None and not columns:
        _matrix(dgate, like, rows, cols, "dgate", dt)
    param = _params(cols, (weight, "weight"), (post_weight, "post_weight"), (gate if columns else None, "gate"))
    grad = _params(cols, (dweight, "dweight"), (dpost_weight, "dpost_weight"), (dgate if columns else None, "dgate"))
    st = (_lib or load()).loco_residual_norm_backward(
        _ptr(dout, dev), _ptr(dh, dev), _ptr(h, dev), _ptr(y, dev), _CODES[x.dtype], _ptr(gate, dev), kind,
        _ptr(post_weight, dev), _ptr(weight, dev), param, _ptr(post_rstd, dev), _ptr(rstd, dev), rows, cols, scale,
        _ptr(dresidual, dev), _ptr(dy, dev), _ptr(dgate, dev), _ptr(dpost_weight, dev), _ptr(dweight, dev), grad,
        _ptr(workspace, dev), _nbytes(workspace), _stream(stream, dev))
    _check("loco_residual_norm_backward", st)


def loco_residual_norm_backward_workspace(rows: int, cols: int) -> int:
    return load().loco_residual_norm_backward_workspace(rows, cols)


# -- log probabilities of tokens ----------------------------------------------------------------

def _runs(shape, strides, what):
    """[(n, step)] of leading dimensions, outermost first, those of one step merged: at most two."""
    runs = []
    for n, s in zip(shape, strides):
        if n == 1:
            continue
        if runs and runs[-1][1] == n * s:
            runs[-1] = (runs[-1][0] * n, s)
        else:
            runs.append((n, s))
    if len(runs) > 2:
        raise ValueError(f"{what}: rows must be one step apart, or sequences of such rows be")
    return runs


def _logits(t, what):
    """(rows, vocab, runs) of a tensor whose last dimension is the vocabulary, each row in one piece; runs as _runs
    gives them, None where the rows follow one another."""
    rows, vocab = _rows_cols(t, what, _FLOATS)
    if rows <= 1 or vocab == 0 or t.is_contiguous():
        if vocab > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what}: a row must be contiguous")
        return rows, vocab, None
    runs = _runs(t.shape[:-1], t.stride()[:-1], what)
    ld = runs[-1][1]
    if ld < vocab or (vocab > 1 and t.stride(-1) != 1):
        raise ValueError(f"{what}: rows must be contiguous and one step of at least {vocab} elements apart")
    if len(runs) == 2 and runs[0][1] < (runs[1][0] - 1) * ld + vocab:
        raise ValueError(f"{what}: sequences must be as far apart as their rows reach")
    return rows, vocab, runs


def _targets(t, rows):
    """The runs of targets that do not follow one another; None for one."""
    if rows <= 1:
        return None
    runs = _runs(t.shape, t.stride(), "targets")
    if len(runs) == 1:  # one target of each sequence
        runs.append((1, 1))
    if runs[-1][1] != 1 or (len(runs) == 2 and runs[0][1] < runs[1][0]):
        raise ValueError("targets must be contiguous, or sequences of them be")
    return runs


def _sequences(rows, *all_runs):
    """(sequences, rows of each, [(step from row to row, from sequence to sequence)]) for each step from row to row of
    buffers that follow one another (an int) or runs."""
    inner = {r[1][0] for r in all_runs if type(r) is not int and len(r) == 2}
    if len(inner) > 1:
        raise ValueError(f"logits, dlogits and targets have sequences of {' and '.join(map(str, sorted(inner)))} rows")
    n = inner.pop() if inner else rows
    steps = []
    for r in all_runs:
        ld = r if type(r) is int else r[-1][1]
        steps.append((ld, r[0][1] if type(r) is not int and len(r) == 2 else n * ld))
    return (rows // n if n else 1), n, steps


def _strided_ptr(t, dev):
    if t is None:
        return None
    d = t.get_device()
    if d != dev:
        if d < 0:
            raise ValueError("tensor must be in device memory")
        raise ValueError(f"tensor is on cuda:{d}; the call runs on the current device, cuda:{dev}")
    return t.data_ptr()


def _row_values(t, like, rows, what, dtypes=_F32) -> None:
    """As _per_row, of other types too."""
    _sized(t, rows, what, dtypes)
    if t is not None and t.dim() > 1 and not _same_rows(tuple(t.shape), tuple(like)[:-1]):
        raise ValueError(f"{what} has the shape {tuple(t.shape)}; the call's is {tuple(like)[:-1]}")


_I64, _I32 = (torch.int64,), (torch.int32,)


def loco_token_logprobs(logits, targets=None, *, logprob=None, entropy=None, stats=None, top_ids=None, top_logprobs=None,
                        scale: float = 1.0, workspace=None, stream=None) -> None:
    """Log probabilities of the targets (int64, one per row; below 0: not scored) under softmax(scale *
    logits) over the last dimension, float32 or bfloat16; the entropy of each row; and its best
    alternatives, top_ids (int32) and top_logprobs (float32), whose last dimension says how many (up to
    LOCO_MAX_TOP), ties to the lower index.  stats (float32, two per row: the largest logit and the
    sum of exp(scale * (logit - it))) is for the backward pass.  Each output is optional.  logits may be a
    slice of wider rows, or of the rows of each sequence, and targets too: logits[:, :-1] with ids[:, 1:].
    workspace: a tensor of token_logprobs_workspace(rows, vocab, top) bytes."""
    dev = _device()
    rows, vocab, runs = _logits(logits, "logits")
    like = logits.shape
    _row_values(targets, like, rows, "targets", _I64)
    _row_values(logprob, like, rows, "logprob")
    _row_values(entropy, like, rows, "entropy")
    _matrix(stats, like, rows, 2, "stats", _F32)
    top = 0
    if top_ids is not None or top_logprobs is not None:
        if top_ids is None or top_logprobs is None or not top_ids.dim():
            raise ValueError("top_ids and top_logprobs go together, with at least one dimension")
        top = top_ids.shape[-1]
        _matrix(top_ids, like, rows, top, "top_ids", _I32)
        _matrix(top_logprobs, like, rows, top, "top_logprobs", _F32)
    truns = None if targets is None or targets.is_contiguous() else _targets(targets, rows)
    seqs, n, ld, seq_ld, target_ld = 1, rows, vocab, 0, 0
    if runs is not None or truns is not None:
        seqs, n, ((ld, seq_ld), (_, target_ld)) = _sequences(rows, runs or vocab, truns or 1)
    st = (_lib or load()).loco_token_logprobs_ex(
        _strided_ptr(logits, dev), _CODES[logits.dtype], seqs, n, vocab, ld, seq_ld, _strided_ptr(targets, dev), target_ld,
        scale, _ptr(logprob, dev), _ptr(entropy, dev), _ptr(stats, dev), top, _ptr(top_ids, dev), _ptr(top_logprobs, dev),
        _ptr(workspace, dev), _nbytes(workspace), _stream(stream, dev))
    _check("loco_token_logprobs", st)


def loco_token_logprobs_workspace(rows: int, vocab: int, top: int = 0) -> int:
    return load().loco_token_logprobs_workspace(rows, vocab, top)


def loco_token_logprobs_backward(logits, targets, stats, *, dlogits, dlogprob=None, entropy=None, dentropy=None,
                                 scale: float = 1.0, stream=None) -> None:
    """dlogits = the gradient of sum(dlogprob * logprob + dentropy * entropy), with stats and entropy as
    loco_token_logprobs wrote them (entropy is needed with dentropy only).  One of dlogprob and dentropy
    may be None.  dlogits has the type and shape of logits, and may be logits itself; each may be a slice as in
    loco_token_logprobs."""
    dev = _device()
    rows, vocab, runs = _logits(logits, "logits")
    like = logits.shape
    drows, dvocab, druns = _logits(dlogits, "dlogits")
    if (drows, dvocab) != (rows, vocab) or not _same_rows(tuple(dlogits.shape[:-1]), tuple(like[:-1])):
        raise ValueError(f"dlogits has the shape {tuple(dlogits.shape)}; the call's is {tuple(like)}")
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits must be {logits.dtype}, not {dlogits.dtype}")
    _row_values(targets, like, rows, "targets", _I64)
    _matrix(stats, like, rows, 2, "stats", _F32)
    for t, what in ((dlogprob, "dlogprob"), (entropy, "entropy"), (dentropy, "dentropy")):
        _row_values(t, like, rows, what)
    truns = None if targets is None or targets.is_contiguous() else _targets(targets, rows)
    seqs, n, ld, seq_ld, dld, dseq_ld, target_ld = 1, rows, vocab, 0, vocab, 0, 0
    if runs is not None or druns is not None or truns is not None:
        seqs, n, ((ld, seq_ld), (dld, dseq_ld), (_, target_ld)) = _sequences(rows, runs or vocab, druns or vocab, truns or 1)
    st = (_lib or load()).loco_token_logprobs_backward_ex(
        _strided_ptr(logits, dev), _CODES[logits.dtype], seqs, n, vocab, ld, seq_ld, _strided_ptr(targets, dev), target_ld,
        scale, _ptr(stats, dev), _ptr(entropy, dev), _ptr(dlogprob, dev), _ptr(dentropy, dev), _strided_ptr(dlogits, dev),
        dld, dseq_ld, _stream(stream, dev))
    _check("loco_token_logprobs_backward", st)


# -- AdamW over many tensors ---------------------------------------------------------------

def _keep(t):
    """The tensor's memory, held for as long as the result lives."""
    return None if t is None else t.detach()


def _alike(t, like, what):
    """t, of as many elements as the shape `like`, must be flat or have that shape: another shape counts
    them in another order."""
    if t is not None and not _same_rows(tuple(t.shape), tuple(like)):
        raise ValueError(f"{what} has the shape {tuple(t.shape)}, not {tuple(like)}")


def _state(state, n, nb, what):
    """(codes or values, exps or None), checked, and the bits of the state."""
    if isinstance(state, torch.Tensor):
        _sized(state, n, what, _F32)
        return state, None, 32
    codes, exps = state
    _sized(codes, n, f"{what} codes", (torch.float8_e4m3fn if what == "m" else torch.uint8,))
    _sized(exps, nb, f"{what} exps", (torch.uint8,))
    return codes, exps, 8


def _stream_of(stream, dev):
    if stream is None:
        return torch.cuda.current_stream(dev)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)


class _Table:
    """Device memory for a table of n tensors, of the stream that fills it: memory that another stream freed may
    still be written by the kernels before."""

    def __init__(self, n, stream, dev):
        nbytes = load().loco_adamw_table_bytes(n)
        self.tensor = self.home = None
        if nbytes:
            s = _stream_of(stream, dev)
            self.home = s.cuda_stream
            with torch.cuda.stream(s):
                self.tensor = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")

    def stream(self, stream, dev):
        """The stream to call on; the memory is not used again before that stream is past the call."""
        handle = _stream(stream, dev)
        if self.tensor is not None and handle != self.home:
            self.tensor.record_stream(_stream_of(stream, dev))
        return handle

    def described(self, stream, dev):
        """Waits until the description is in the table: a step on another stream may follow at once, and would
        take what it read before for addresses."""
        if self.tensor is not None:
            _stream_of(stream, dev).synchronize()


def _not_captured():
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("describe the tensors before a graph is captured: the table is filled on the device")


class AdamwTensors:
    """The tensors of loco_adamw, checked and described once; a training loop keeps it from step to
    step.  tensors: an iterable of (param, grad, m, v[, param_bf16[, weight_decay]]): param
    float32 or bfloat16, grad float32 or bfloat16, m and v float32, or in 8 bits (m: (codes
    float8_e4m3fn, exps uint8), v: (codes uint8, exps uint8), one exps byte per block); every
    param, every grad and every state of one kind; grad and param_bf16 flat or of the param's
    shape.  param_bf16 (or None) receives the bfloat16 copy of a float32 param.  weight_decay is that
    of the tensors that do not give one.  The memory of the tensors is kept alive and must not be resized; later calls use it as it is now, on the
    device that is current now.  The description is on the device when the constructor returns; it
    cannot be made while a graph is captured, and has to live as long as a graph that steps it."""

    def __init__(self, tensors, *, block: int = 256, weight_decay: float = 0.0, stream=None, _wait: bool = True):
        self.device, self.block = _device(), block
        dev, rows, keep = self.device, [], []
        self.param_dtype = self.grad_dtype = self.bits = None
        self.told = False  # that 8-bit states want a seed
        for i, t in enumerate(tensors):
            if not 4 <= len(t) <= 6:
                raise ValueError(f"tensor {i}: expected (param, grad, m, v[, param_bf16[, weight_decay]])")
            param, grad, m, v, copy, decay = (*t, None, None)[:6]
            if param.dtype not in _CODES or grad.dtype not in _CODES:
                raise TypeError(f"tensor {i}: param and grad must be float32 or bfloat16")
            n = param.numel()
            nb = num_blocks(n, block) if block > 0 else 0
            _sized(grad, n, f"tensor {i}: grad", _FLOATS)
            m, me, bits = _state(m, n, nb, "m")
            v, ve, vbits = _state(v, n, nb, "v")
            kind = (param.dtype, grad.dtype, bits)
            if vbits != bits or (i and kind != (self.param_dtype, self.grad_dtype, self.bits)):
                raise TypeError(f"tensor {i}: all params, grads and states must be of one kind")
            self.param_dtype, self.grad_dtype, self.bits = kind
            if copy is not None and param.dtype != torch.float32:
                raise TypeError(f"tensor {i}: param_bf16 goes with a float32 param")
            _sized(copy, n, f"tensor {i}: param_bf16", _BF)
            _alike(grad, param.shape, f"tensor {i}: grad")
            _alike(copy, param.shape, f"tensor {i}: param_bf16")
            parts = (param, grad, m, v, me, ve, copy)
            rows.append((*(_ptr(x, dev) for x in parts), n, weight_decay if decay is None else decay))
            keep.append(tuple(_keep(x) for x in parts))
        count = len(rows)
        if _wait and count:
            _not_captured()
        array = (AdamwTensor * max(1, count))(*(AdamwTensor(*r) for r in rows))
        table = _Table(count, stream, dev)
        self._keep, self._table, self.plan = (keep, array), table, AdamwPlan()
        st = load().loco_adamw_plan(array, count, _CODES.get(self.param_dtype, LOCO_F32),
                                    _CODES.get(self.grad_dtype, LOCO_F32), self.bits or 32, block, _ptr(table.tensor, dev),
                                    _nbytes(table.tensor), ctypes.byref(self.plan), table.stream(stream, dev))
        _check("loco_adamw_plan", st)
        if _wait:
            table.described(stream, dev)


def loco_adamw(tensors, *, step: int, lr: float, beta1: float = 0.9, beta2: float | None = None, eps: float = 1e-8,
               weight_decay: float | None = None, block: int | None = None, grad_scale=None, seed=None,
               stream=None) -> None:
    """One AdamW step (decoupled weight decay, bias correction) of all tensors.  tensors: an
    AdamwTensors, which has its own block and weight_decay, or what its constructor takes.  beta1
    and beta2 (None: 0.999) are the weights of the old moments; step counts from 1; grad_scale is a
    float32 tensor of one element, or None.  lr, step and the others are read during the call: a
    captured graph repeats them.

    seed: an int, or an int64 tensor of one element.  With it, 8-bit states are rounded at random, by bits
    that seed, step and the element's place among the tensors decide, and follow their averages over a
    run.  It may stay the same from step to step; ranks that hold copies of the tensors take the same
    one, other lists of tensors another.  A captured graph, which repeats step, needs a tensor that the
    graph raises at each replay.  Without a seed 8-bit states are rounded to nearest, for a single step:
    over many, a state that changes by less than half a step of its code at once stays where it is.
    Then beta2 has no default, and the first such step of a description warns."""
    if not isinstance(tensors, AdamwTensors):
        tensors = AdamwTensors(tensors, block=256 if block is None else block, weight_decay=weight_decay or 0.0,
                               stream=stream, _wait=False)
    elif block is not None or weight_decay is not None:
        raise ValueError("an AdamwTensors has its own block and weight_decay")
    dev = _device()
    if dev != tensors.device:
        raise ValueError(f"the tensors are on cuda:{tensors.device}; the call runs on the current device, cuda:{dev}")
    _sized(grad_scale, 1, "grad_scale", _F32)
    rounding = None
    if seed is None:
        if tensors.bits == 8:
            if beta2 is None:
                raise ValueError("8-bit states need a seed: rounded to nearest they do not follow their averages "
                                 "(for a single step without one, give beta2)")
            if not tensors.told:
                tensors.told = True
                warnings.warn("8-bit states are rounded to nearest without a seed: over many steps they do not follow "
                              "their averages", RuntimeWarning, stacklevel=2)
    elif isinstance(seed, torch.Tensor):
        _sized(seed, 1, "seed", _I64)
        rounding = ctypes.byref(AdamwRounding(0, _ptr(seed, dev)))
    else:
        rounding = ctypes.byref(AdamwRounding(operator.index(seed) & 0xFFFFFFFFFFFFFFFF, None))
    opt = AdamwOptions(lr, beta1, 0.999 if beta2 is None else beta2, eps, step)
    st = (_lib or load()).loco_adamw_ex(ctypes.byref(tensors.plan), ctypes.byref(opt), _ptr(grad_scale, dev), rounding,
                                        tensors._table.stream(stream, dev))
    _check("loco_adamw", st)


class AdamwStates:
    """8-bit states and the tensors of their values, checked and described once.  states: an
    iterable of ((codes, exps), values), values float32 or bfloat16, all alike; codes in
    float8_e4m3fn are a first moment, in uint8 a second one.  Memory and device as in AdamwTensors."""

    def __init__(self, states, *, block: int = 256, stream=None, _wait: bool = True):
        self.device, self.block, self.dtype = _device(), block, None
        dev, rows, keep = self.device, [], []
        for i, ((codes, exps), values) in enumerate(states):
            n = codes.numel()
            if codes.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise TypeError(f"state {i}: codes must be float8_e4m3fn or uint8, not {codes.dtype}")
            _sized(exps, num_blocks(n, block) if block > 0 else 0, f"state {i}: exps", (torch.uint8,))
            _sized(values, n, f"state {i}: values", _FLOATS if i == 0 else (self.dtype,))
            self.dtype = values.dtype
            rows.append((_ptr(codes, dev), _ptr(exps, dev), _ptr(values, dev), n,
                         1 if codes.dtype == torch.float8_e4m3fn else 2))
            keep.append((_keep(codes), _keep(exps), _keep(values)))
        count = len(rows)
        if _wait and count:
            _not_captured()
        array = (AdamwState * max(1, count))(*(AdamwState(*r) for r in rows))
        table = _Table(count, stream, dev)
        self._keep, self._table, self.plan = keep, table, AdamwPlan()
        st = load().loco_adamw_state_plan(array, count, block, _CODES.get(self.dtype, LOCO_F32), _ptr(table.tensor, dev),
                                          _nbytes(table.tensor), ctypes.byref(self.plan), table.stream(stream, dev))
        _check("loco_adamw_state_plan", st)
        if _wait:
            table.described(stream, dev)


def _adamw_states(name, states, block, stream):
    if not isinstance(states, AdamwStates):
        states = AdamwStates(states, block=256 if block is None else block, stream=stream, _wait=False)
    elif block is not None:
        raise ValueError("an AdamwStates has its own block")
    dev = _device()
    if dev != states.device:
        raise ValueError(f"the states are on cuda:{states.device}; the call runs on the current device, cuda:{dev}")
    _check(name, getattr(_lib or load(), name)(ctypes.byref(states.plan), states._table.stream(stream, dev)))


def loco_adamw_state_read(states, *, block: int | None = None, stream=None) -> None:
    """values = what the 8-bit states stand for, exactly.  states: an AdamwStates, or what its
    constructor takes."""
    _adamw_states("loco_adamw_state_read", states, block, stream)


def loco_adamw_state_write(states, *, block: int | None = None, stream=None) -> None:
    """The 8-bit states of the values, rounded as loco_adamw rounds them."""
    _adamw_states("loco_adamw_state_write", states, block, stream)


# short names
compensate_quantize = loco_compensate_quantize
compensate_quantize_ex = loco_compensate_quantize_ex
dequant_reduce = loco_dequant_reduce
dequant_reduce_adam = loco_dequant_reduce_adam
topk_quantize = loco_topk_quantize
sparse_aggregate = loco_sparse_aggregate
layer_norm = loco_layer_norm
layer_norm_backward = loco_layer_norm_backward
layer_norm_backward_workspace = loco_layer_norm_backward_workspace
checkpoint_write = loco_checkpoint_write
checkpoint_read = loco_checkpoint_read
linear = loco_linear
linear_workspace = loco_linear_workspace
linear_input_grad = loco_linear_input_grad
linear_input_grad_workspace = loco_linear_input_grad_workspace
linear_weight_grad = loco_linear_weight_grad
linear_weight_grad_workspace = loco_linear_weight_grad_workspace
adamw = loco_adamw
adamw_state_read = loco_adamw_state_read
adamw_state_write = loco_adamw_state_write
residual_norm = loco_residual_norm
residual_norm_backward = loco_residual_norm_backward
residual_norm_backward_workspace = loco_residual_norm_backward_workspace
token_logprobs = loco_token_logprobs
token_logprobs_workspace = loco_token_logprobs_workspace
token_logprobs_backward = loco_token_logprobs_backward
