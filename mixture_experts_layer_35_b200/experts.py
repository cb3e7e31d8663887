"""Expert operators: the steps between ``moe.permute`` and the layer's output one by one,
with their gradients and with 8-bit operands (declared in include/moe.h).

A run of them, for logits of M tokens and 8-bit weights::

    w, ids, _ = moe.router_topk(logits, K)
    offsets, perm, inv = moe.permute(ids, E)
    xq, xs = experts.dispatch_quantize(x, inv)
    hq, hs = experts.product_activation(xq, xs, w13_q, w13_s, offsets, "swiglu")
    y = experts.combine(experts.product(hq, hs, w2_q, w2_s, offsets), inv, w)

Argument marshalling only, as in ``moe``: every operator is one CUDA kernel of libmoe.so.
Tensors must be contiguous, 16-byte aligned and all on one CUDA device, which need not be
the current one; a wrong type, shape, device or layout raises ValueError before anything
is launched, and a refusal by the library raises ``moe.MoEError``.  Work and new outputs belong to
``stream`` (default: the device's current stream); inputs must be ready there, and must not be freed for
another stream before that work is done.

Nothing is recorded for autograd: an input that requires grad is read as data, no output requires grad, and a
write to ``out`` is not counted as a change.  Gradients are calls of their own (``*_backward``, ``*_grad``), to
be made by the training step or from a ``torch.autograd.Function``.
"""
from __future__ import annotations

import ctypes
import operator
from typing import Optional

import torch

from . import moe
from .moe import ACT, MOE_ERR_DEVICE, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_OK, MoEError, _lib

BLOCK = 128  # MOE_QUANT_BLOCK
MAX_ROWS = 65536 * 8  # MOE_MAX_ROWS
DTYPES = {torch.bfloat16: moe.DT_BF16, torch.float32: moe.DT_FP32}
FP8 = {torch.float8_e4m3fn: moe.DT_E4M3, torch.float8_e5m2: moe.DT_E5M2}

_vp, _ci = ctypes.c_void_p, ctypes.c_int
for _name, _args in (
        ("moe_dispatch", [_vp, _ci, _ci, _ci, _ci, _vp, _ci, _vp, _vp]),
        ("moe_combine", [_vp, _ci, _ci, _ci, _ci, _vp, _ci, _vp, _vp, _vp]),
        ("moe_combine_backward", [_vp, _vp, _ci, _ci, _ci, _ci, _vp, _ci, _vp, _vp, _vp, _vp]),
        ("moe_quantize_rows", [_vp, _ci, _ci, _ci, _ci, _vp, _vp, _vp]),
        ("moe_dispatch_quantize", [_vp, _ci, _ci, _ci, _ci, _vp, _ci, _ci, _vp, _vp, _vp]),
        ("moe_quantize_blocks", [_vp, _ci, _ci, _ci, _ci, _ci, _vp, _vp, _vp]),
        ("moe_column_blocks", [_ci, _ci]),
        ("moe_quantize_columns", [_vp, _ci, _ci, _ci, _vp, _ci, _ci, _vp, _vp, _vp]),
        ("moe_activation", [_vp, _ci, _ci, _ci, _ci, _vp, _vp]),
        ("moe_activation_quantize", [_vp, _ci, _ci, _ci, _ci, _ci, _vp, _vp, _vp]),
        ("moe_activation_backward", [_vp, _vp, _ci, _ci, _ci, _ci, _vp, _vp]),
        ("moe_product", [_vp, _vp, _ci, _vp, _vp, _ci, _ci, _ci, _vp, _ci, _ci, _vp, _vp]),
        ("moe_product_activation", [_vp, _vp, _ci, _vp, _vp, _ci, _ci, _ci, _vp, _ci, _ci, _ci, _vp, _vp, _vp]),
        ("moe_product_input_grad", [_vp, _vp, _ci, _vp, _vp, _ci, _ci, _ci, _vp, _ci, _ci, _vp, _vp]),
        ("moe_product_weight_grad", [_vp, _vp, _ci, _vp, _vp, _ci, _ci, _ci, _ci, _vp, _ci, _ci, _ci, _vp, _vp]),
        ("moe_product_get_error", [ctypes.POINTER(_ci), _vp])):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _ci


# ---------------------------------------------------------------- checks
def _tensor(name: str, t, device, dtypes, shape):
    """``t`` is a contiguous tensor of one of ``dtypes`` and of ``shape`` (None: any) on ``device``."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    got = t.shape
    if got != shape and (len(got) != len(shape) or any(n is not None and n != m for n, m in zip(shape, got))):
        raise ValueError(f"{name}: expected shape {tuple('any' if n is None else n for n in shape)}, got {tuple(got)}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def _narrow(name: str, t):
    """``t``'s sizes fit the library's 32-bit arguments."""
    if t.dim() and max(t.shape) >> 31:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} of shape {tuple(t.shape)}")


def _first(name: str, t):
    """The device of an operator's first tensor."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    n = t.numel()
    if n >> 31 or n == 0:
        _narrow(name, t)
    return t.device


def _count(name: str, n, most: int) -> int:
    """A number of rows or tokens, at most ``most``."""
    try:
        n = operator.index(n)
    except TypeError:
        raise ValueError(f"{name}: expected a whole number, got {type(n).__name__}") from None
    if not 0 <= n <= most:
        raise MoEError(MOE_ERR_INVALID_ARG if n < 0 else MOE_ERR_UNSUPPORTED, f"{name} {n}")
    return n


def _key(table: dict, key, what: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{what}: expected {' or '.join(str(k) for k in table)}, got {key}") from None


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


# The current stream's handle without building a torch.cuda.Stream (0.1 against 2.3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """Makes ``device`` current, and ``stream`` when one is given, for the outputs' allocation and the
    launch; entering gives the stream's handle."""
    __slots__ = ("_guards", "_stream", "_device")

    def __init__(self, device, stream):
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                try:
                    stream = torch.cuda.ExternalStream(operator.index(stream), device=device)
                except TypeError:
                    raise ValueError(f"stream: expected a stream or its handle, got {type(stream).__name__}") from None
            if stream.device != device:
                raise ValueError(f"stream: expected one of {device}, got one of {stream.device}")
        self._guards, self._stream, self._device = (), stream, device

    def __enter__(self):
        device, stream = self._device, self._stream
        if stream is not None:
            self._guards = (torch.cuda.stream(stream),)  # makes its device current too
        elif torch.cuda.current_device() != device.index:
            self._guards = (torch.cuda.device(device),)
        for g in self._guards:
            g.__enter__()
        return _raw_stream(device.index) if stream is None else stream.cuda_stream

    def __exit__(self, *exc):
        for g in self._guards:
            g.__exit__(*exc)


def _out(name, out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _tensor(name, out, device, (dtype,), shape)


def _pair(out):
    if out is None:
        return None, None
    if not isinstance(out, (tuple, list)) or len(out) != 2:
        raise ValueError("out: expected two tensors")
    return out


def _call(name: str, *args):
    st = getattr(_lib, name)(*args)
    if st != MOE_OK:
        raise MoEError(st, name)


def _slots(inv, M: int, device):
    _tensor("inv", inv, device, (torch.int32,), (None,))
    n = inv.numel()
    if n >> 31:
        _narrow("inv", inv)
    if M == 0:
        if n:
            raise ValueError("inv: expected no slots for no tokens")
        return 1
    if n == 0 or n % M:
        raise ValueError(f"inv: expected a multiple of {M} slots, got {n}")
    return n // M


def _experts(offsets) -> int:
    """The number of experts that offsets (None: one expert) belong to."""
    if offsets is None:
        return 1
    if not isinstance(offsets, torch.Tensor):
        raise ValueError(f"offsets: expected a tensor, got {type(offsets).__name__}")
    _narrow("offsets", offsets)
    return max(1, offsets.numel() - 1)


def _offsets(offsets, E: int, device):
    if offsets is None:
        if E != 1:
            raise ValueError(f"offsets: needed for {E} experts")
        return None
    return _tensor("offsets", offsets, device, (torch.int32,), (E + 1,)).data_ptr()


# ---------------------------------------------------------------- rows
def dispatch(x: torch.Tensor, inv: torch.Tensor, rows: Optional[int] = None, out=None, stream=None):
    """Tokens [M, H] to their experts' rows [rows, H] (moe_dispatch); ``inv`` as ``moe.permute`` gives it.
    ``rows``: the number of rows, len(inv) by default; slots whose row is outside are dropped."""
    dev = _first("x", x)
    _tensor("x", x, dev, DTYPES, (None, None))
    M, H = x.shape
    K = _slots(inv, M, dev)
    P = inv.numel() if rows is None else _count("rows", rows, MAX_ROWS)
    with _On(dev, stream) as s:
        out = _out("out", out, (P, H), x.dtype, dev)
        _call("moe_dispatch", x.data_ptr(), DTYPES[x.dtype], M, K, H, inv.data_ptr(), P, out.data_ptr(), s)
    return out


def dispatch_backward(dxs: torch.Tensor, inv: torch.Tensor, M: int, out=None, stream=None):
    """Gradient of ``dispatch``: rows [P, H] summed per token into [M, H]."""
    return _combine(dxs, inv, None, _count("M", M, MAX_ROWS), out, stream)


def dispatch_quantize(x: torch.Tensor, inv: torch.Tensor, rows: Optional[int] = None,
                      dtype: torch.dtype = torch.float8_e4m3fn, out=None, stream=None):
    """``dispatch`` to 8-bit rows with one scale per 128 columns (moe_dispatch_quantize):
    ([rows, H] of ``dtype``, [rows, ceil(H / 128)] FP32)."""
    dev = _first("x", x)
    _tensor("x", x, dev, DTYPES, (None, None))
    fp8 = _key(FP8, dtype, "dtype")
    M, H = x.shape
    K = _slots(inv, M, dev)
    P = inv.numel() if rows is None else _count("rows", rows, MAX_ROWS)
    q, sc = _pair(out)
    with _On(dev, stream) as s:
        q = _out("out[0]", q, (P, H), dtype, dev)
        sc = _out("out[1]", sc, (P, _blocks(H)), torch.float32, dev)
        _call("moe_dispatch_quantize", x.data_ptr(), DTYPES[x.dtype], M, K, H, inv.data_ptr(), P, fp8, q.data_ptr(),
              sc.data_ptr(), s)
    return q, sc


def _combine(ys, inv, weights, M, out, stream):
    dev = _first("ys", ys)
    _tensor("ys", ys, dev, DTYPES, (None, None))
    P, H = ys.shape
    K = _slots(inv, M, dev)
    if weights is not None:
        _tensor("weights", weights, dev, (torch.float32,), (M, K if M else None))
    with _On(dev, stream) as s:
        out = _out("out", out, (M, H), ys.dtype, dev)
        _call("moe_combine", ys.data_ptr(), DTYPES[ys.dtype], M, K, H, inv.data_ptr(), P,
              None if weights is None else weights.data_ptr(), out.data_ptr(), s)
    return out


def combine(ys: torch.Tensor, inv: torch.Tensor, weights: torch.Tensor, out=None, stream=None):
    """The experts' rows [P, H] weighted by [M, K] and summed per token into [M, H] (moe_combine)."""
    _first("weights", weights)
    if weights.dim() != 2:
        raise ValueError(f"weights: expected two dimensions, got {weights.dim()}")
    return _combine(ys, inv, weights, weights.shape[0], out, stream)


def combine_backward(dy: torch.Tensor, ys: torch.Tensor, inv: torch.Tensor, weights: torch.Tensor, out=None,
                     stream=None):
    """Gradients of ``combine`` from dy [M, H]: (of the rows [P, H], of the weights [M, K])
    (moe_combine_backward)."""
    dev = _first("dy", dy)
    _tensor("dy", dy, dev, DTYPES, (None, None))
    M, H = dy.shape
    _tensor("ys", ys, dev, (dy.dtype,), (None, H))
    _narrow("ys", ys)
    K = _slots(inv, M, dev)
    _tensor("weights", weights, dev, (torch.float32,), (M, K if M else None))
    dys, dw = _pair(out)
    with _On(dev, stream) as s:
        dys = _out("out[0]", dys, tuple(ys.shape), dy.dtype, dev)
        dw = _out("out[1]", dw, tuple(weights.shape), torch.float32, dev)
        _call("moe_combine_backward", dy.data_ptr(), ys.data_ptr(), DTYPES[dy.dtype], M, K, H, inv.data_ptr(),
              ys.shape[0], weights.data_ptr(), dys.data_ptr(), dw.data_ptr(), s)
    return dys, dw


# ---------------------------------------------------------------- 8-bit blocks
def quantize_rows(x: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, out=None, stream=None):
    """[R, C] to 8 bits with one scale per row and 128 columns (moe_quantize_rows):
    ([R, C] of ``dtype``, [R, ceil(C / 128)] FP32)."""
    dev = _first("x", x)
    _tensor("x", x, dev, DTYPES, (None, None))
    fp8 = _key(FP8, dtype, "dtype")
    R, C = x.shape
    q, sc = _pair(out)
    with _On(dev, stream) as s:
        q = _out("out[0]", q, (R, C), dtype, dev)
        sc = _out("out[1]", sc, (R, _blocks(C)), torch.float32, dev)
        _call("moe_quantize_rows", x.data_ptr(), DTYPES[x.dtype], R, C, fp8, q.data_ptr(), sc.data_ptr(), s)
    return q, sc


def quantize_blocks(w: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, out=None, stream=None):
    """Weights [E, N, C] to 8 bits with one scale per 128 x 128 block (moe_quantize_blocks):
    ([E, N, C] of ``dtype``, [E, ceil(N / 128), ceil(C / 128)] FP32)."""
    dev = _first("w", w)
    _tensor("w", w, dev, DTYPES, (None, None, None))
    fp8 = _key(FP8, dtype, "dtype")
    E, N, C = w.shape
    q, sc = _pair(out)
    with _On(dev, stream) as s:
        q = _out("out[0]", q, (E, N, C), dtype, dev)
        sc = _out("out[1]", sc, (E, _blocks(N), _blocks(C)), torch.float32, dev)
        _call("moe_quantize_blocks", w.data_ptr(), DTYPES[w.dtype], E, N, C, fp8, q.data_ptr(), sc.data_ptr(), s)
    return q, sc


def column_blocks(P: int, E: int) -> int:
    """128-row blocks that hold P rows of E experts, however they are split (moe_column_blocks)."""
    return _lib.moe_column_blocks(P, E)


def quantize_columns(x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                     dtype: torch.dtype = torch.float8_e4m3fn, out=None, stream=None):
    """[P, C] to 8 bits with one scale per column and 128 rows of an expert (moe_quantize_columns):
    ([B * 128, C] of ``dtype``, [B, C] FP32) with B = column_blocks(P, E); blocks behind the last
    expert's are left as they were (without offsets: zeros).  Offsets may name more rows than the P
    that there are: blocks of rows that are not there are zeros."""
    dev = _first("x", x)
    _tensor("x", x, dev, DTYPES, (None, None))
    fp8 = _key(FP8, dtype, "dtype")
    P, C = x.shape
    E = _experts(offsets)
    off = _offsets(offsets, E, dev)
    B = column_blocks(P, E)
    q, sc = _pair(out)
    with _On(dev, stream) as s:
        q = _out("out[0]", q, (B * BLOCK, C), dtype, dev)
        sc = _out("out[1]", sc, (B, C), torch.float32, dev)
        _call("moe_quantize_columns", x.data_ptr(), DTYPES[x.dtype], P, C, off, E, fp8, q.data_ptr(), sc.data_ptr(), s)
    return q, sc


# ---------------------------------------------------------------- activation
def _features(y, act: str) -> int:
    n = y.shape[1]
    if act == "swiglu":
        if n % 2:
            raise ValueError(f"y: SwiGLU needs an even number of columns, got {n}")
        return n // 2
    return n


def activation(y: torch.Tensor, act: str, out=None, stream=None):
    """SwiGLU of [P, 2I] (gate, up) or ReLU^2 of [P, I] to [P, I] (moe_activation)."""
    dev = _first("y", y)
    _tensor("y", y, dev, DTYPES, (None, None))
    a = _key(ACT, act, "act")
    I = _features(y, act)
    with _On(dev, stream) as s:
        out = _out("out", out, (y.shape[0], I), y.dtype, dev)
        _call("moe_activation", y.data_ptr(), DTYPES[y.dtype], a, y.shape[0], I, out.data_ptr(), s)
    return out


def activation_quantize(y: torch.Tensor, act: str, dtype: torch.dtype = torch.float8_e4m3fn, out=None, stream=None):
    """``activation`` and ``quantize_rows`` of its FP32 values (moe_activation_quantize)."""
    dev = _first("y", y)
    _tensor("y", y, dev, DTYPES, (None, None))
    a, fp8 = _key(ACT, act, "act"), _key(FP8, dtype, "dtype")
    P, I = y.shape[0], _features(y, act)
    q, sc = _pair(out)
    with _On(dev, stream) as s:
        q = _out("out[0]", q, (P, I), dtype, dev)
        sc = _out("out[1]", sc, (P, _blocks(I)), torch.float32, dev)
        _call("moe_activation_quantize", y.data_ptr(), DTYPES[y.dtype], a, P, I, fp8, q.data_ptr(), sc.data_ptr(), s)
    return q, sc


def activation_backward(y: torch.Tensor, dh: torch.Tensor, act: str, out=None, stream=None):
    """Gradient of ``activation`` with respect to y, from dh [P, I] (moe_activation_backward)."""
    dev = _first("y", y)
    _tensor("y", y, dev, DTYPES, (None, None))
    a = _key(ACT, act, "act")
    I = _features(y, act)
    _tensor("dh", dh, dev, (y.dtype,), (y.shape[0], I))
    with _On(dev, stream) as s:
        out = _out("out", out, tuple(y.shape), y.dtype, dev)
        _call("moe_activation_backward", y.data_ptr(), dh.data_ptr(), DTYPES[y.dtype], a, y.shape[0], I,
              out.data_ptr(), s)
    return out


# ---------------------------------------------------------------- products
def _operands(names, q, sc, wq, ws, offsets, columns: int):
    """Checks of a row operand and the weights; (device, P, E, N, C, offsets pointer).
    ``columns``: the weights' dimension that the row operand's columns match."""
    dev = _first(names[0], q)
    _tensor("wq", wq, dev, (torch.float8_e4m3fn,), (None, None, None))
    E, N, C = wq.shape
    if (E | N | C) >> 31:
        _narrow("wq", wq)
    _tensor("ws", ws, dev, (torch.float32,), (E, _blocks(N), _blocks(C)))
    _tensor(names[0], q, dev, FP8, (None, wq.shape[columns]))
    _tensor(names[1], sc, dev, (torch.float32,), (q.shape[0], _blocks(q.shape[1])))
    return dev, q.shape[0], E, N, C, _offsets(offsets, E, dev)


def product(xq, xs, wq, ws, offsets: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
            out=None, stream=None):
    """Each row times its expert's weights, [P, C] x [E, N, C] -> [P, N] (moe_product).  ``xq``, ``xs``: from
    ``quantize_rows`` or ``dispatch_quantize``; ``wq`` (e4m3), ``ws``: from ``quantize_blocks``."""
    dev, P, E, N, C, off = _operands(("xq", "xs"), xq, xs, wq, ws, offsets, 2)
    dt = _key(DTYPES, out_dtype, "out_dtype")
    with _On(dev, stream) as s:
        out = _out("out", out, (P, N), out_dtype, dev)
        _call("moe_product", xq.data_ptr(), xs.data_ptr(), FP8[xq.dtype], wq.data_ptr(), ws.data_ptr(), P, N, C, off,
              E, dt, out.data_ptr(), s)
    return out


def product_activation(xq, xs, wq, ws, offsets: Optional[torch.Tensor] = None, act: str = "swiglu",
                       dtype: torch.dtype = torch.float8_e4m3fn, out=None, stream=None):
    """``product``, ``activation`` and ``quantize_rows`` in one kernel (moe_product_activation): wq [E, 2I, C]
    (swiglu: gate rows, then up rows) or [E, I, C] (relu2) -> ([P, I] of ``dtype``, [P, ceil(I / 128)] FP32)."""
    dev, P, E, N, C, off = _operands(("xq", "xs"), xq, xs, wq, ws, offsets, 2)
    a, fp8 = _key(ACT, act, "act"), _key(FP8, dtype, "dtype")
    if act == "swiglu" and N % 2:
        raise ValueError(f"wq: SwiGLU needs an even number of rows, got {N}")
    I = N // 2 if act == "swiglu" else N
    q, sc = _pair(out)
    with _On(dev, stream) as s:
        q = _out("out[0]", q, (P, I), dtype, dev)
        sc = _out("out[1]", sc, (P, _blocks(I)), torch.float32, dev)
        _call("moe_product_activation", xq.data_ptr(), xs.data_ptr(), FP8[xq.dtype], wq.data_ptr(), ws.data_ptr(), P,
              I, C, off, E, a, fp8, q.data_ptr(), sc.data_ptr(), s)
    return q, sc


def product_input_grad(dyq, dys, wq, ws, offsets: Optional[torch.Tensor] = None,
                       out_dtype: torch.dtype = torch.bfloat16, out=None, stream=None):
    """Gradient of ``product`` with respect to its rows, [P, N] x [E, N, C] -> [P, C]
    (moe_product_input_grad), from the same weights; ``dyq``, ``dys``: from ``quantize_rows``."""
    dev, P, E, N, C, off = _operands(("dyq", "dys"), dyq, dys, wq, ws, offsets, 1)
    dt = _key(DTYPES, out_dtype, "out_dtype")
    with _On(dev, stream) as s:
        out = _out("out", out, (P, C), out_dtype, dev)
        _call("moe_product_input_grad", dyq.data_ptr(), dys.data_ptr(), FP8[dyq.dtype], wq.data_ptr(), ws.data_ptr(),
              P, N, C, off, E, dt, out.data_ptr(), s)
    return out


def product_weight_grad(dyq, dys, xq, xs, offsets: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                        out=None, accumulate: bool = False, stream=None):
    """Gradient of ``product`` with respect to its weights, [E, N, C] (moe_product_weight_grad); the operands
    from ``quantize_columns`` of dy [P, N] and x [P, C] with these offsets.  ``accumulate``: add to ``out``."""
    dev = _first("dyq", dyq)
    _tensor("dyq", dyq, dev, FP8, (None, None))
    B, N = dyq.shape[0] // BLOCK, dyq.shape[1]
    if dyq.shape[0] != B * BLOCK:
        raise ValueError(f"dyq: expected a multiple of {BLOCK} rows, got {dyq.shape[0]}")
    _tensor("dys", dys, dev, (torch.float32,), (B, N))
    _tensor("xq", xq, dev, FP8, (B * BLOCK, None))
    _narrow("xq", xq)
    C = xq.shape[1]
    _tensor("xs", xs, dev, (torch.float32,), (B, C))
    E = _experts(offsets)
    off = _offsets(offsets, E, dev)
    dt = _key(DTYPES, out_dtype, "out_dtype")
    if accumulate and out is None:
        raise ValueError("out: needed to accumulate")
    with _On(dev, stream) as s:
        out = _out("out", out, (E, N, C), out_dtype, dev)
        _call("moe_product_weight_grad", dyq.data_ptr(), dys.data_ptr(), FP8[dyq.dtype], xq.data_ptr(), xs.data_ptr(),
              FP8[xq.dtype], B, N, C, off, E, dt, int(bool(accumulate)), out.data_ptr(), s)
    return out


def get_error(stream=None) -> int:
    """Read and clear the products' device error word of the current device (moe_product_get_error)."""
    code = _ci(0)
    st = _lib.moe_product_get_error(ctypes.byref(code), moe._stream(stream))
    if st not in (MOE_OK, MOE_ERR_DEVICE):
        raise MoEError(st, "moe_product_get_error")
    return code.value
