"""Python binding of libloco.so (ctypes): argument marshalling only.

Every function takes torch tensors (device memory) and passes their pointers, sizes and
the current HIP stream to the C ABI of the same name; every step of the computation
runs in the library's HIP kernels.  There is no fallback: if the library is missing or
a call returns an error status, the call raises.
"""

from __future__ import annotations

import ctypes
import math
import os

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

SYMBOLS = ["loco_compensate_quantize", "loco_compensate_quantize_ex", "loco_dequant_reduce",
           "loco_dequant_reduce_adam", "loco_topk_quantize", "loco_sparse_aggregate", "loco_status_string",
           "loco_version", "loco_layer_norm", "loco_layer_norm_backward", "loco_layer_norm_backward_workspace",
           "loco_checkpoint_write", "loco_checkpoint_read", "loco_linear", "loco_linear_workspace",
           "loco_linear_input_grad", "loco_linear_input_grad_workspace", "loco_linear_weight_grad",
           "loco_linear_weight_grad_workspace"]


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
            ("loco_linear_weight_grad_workspace", i64, [i64, i64, i64, i32])):
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
