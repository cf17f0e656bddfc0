"""Python binding of the int8 products with token and channel scales, dense and
grouped by expert, and of the row quantisation, expert positions and combine
that go with them (include/llmint8.h).

Argument marshalling only, as llmint8.py: dtypes, shapes, devices and layouts
are checked, outputs that are not given are allocated on the call's stream, and
the library's kernels do the rest.  Calls run on the device of their tensors,
whichever is current.
"""
from __future__ import annotations

import ctypes

import torch

from .llmint8 import _check, _need, llmint8_quantize_weight, load_library

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
MAX_EXPERTS = 1024


def _same_device(first: torch.Tensor, **others):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _shape(t: torch.Tensor, shape: tuple, name: str):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _float(t, ndim: int, name: str):
    if isinstance(t, torch.Tensor) and t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    _need(t, t.dtype if isinstance(t, torch.Tensor) else None, ndim, name)


def _out_dtype(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
    return _DTYPES[dtype]


class _On:
    """The tensors' device and the call's stream, current while outputs are
    allocated and kernels launched (an output belongs to the stream that
    writes it)."""

    __slots__ = ("guard", "stream")

    def __init__(self, device: torch.device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self.guard = None
        if stream is not None:
            self.guard = torch.cuda.stream(stream)
        elif device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)
            stream = torch.cuda.current_stream(device)
        else:
            stream = torch.cuda.current_stream()
        self.stream = stream.cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return ctypes.c_void_p(self.stream)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def llmint8_quantize_rows(X: torch.Tensor, positions: torch.Tensor | None = None, Xq: torch.Tensor | None = None,
                          xscale: torch.Tensor | None = None, stream=None):
    """X [T, K] (float16, bfloat16 or float32) -> (Xq int8, xscale float32), one
    scale per row: max|x| / 127.

    With positions (int32 [T, k], llmint8_expert_positions) row t is written to
    every row positions[t, j] >= 0 of Xq [S, K] and xscale [S]; S is T k unless
    Xq is given, and rows that no position names are left as they were.
    Positions must be distinct.  A row with a NaN or an infinity gets the scale
    NaN and codes 0."""
    _float(X, 2, "X")
    T, K = X.shape
    copies = 0
    S = T
    if positions is not None:
        _need(positions, torch.int32, 2, "positions")
        copies = positions.shape[1]
        _shape(positions, (T, copies), "positions")
        if copies < 1:
            raise ValueError("positions must have a column")
        S = T * copies if Xq is None else Xq.shape[0]
    with _On(X.device, stream) as st:
        Xq = torch.empty((S, K), dtype=torch.int8, device=X.device) if Xq is None else Xq
        xscale = torch.empty(S, dtype=torch.float32, device=X.device) if xscale is None else xscale
        _need(Xq, torch.int8, 2, "Xq")
        _need(xscale, torch.float32, 1, "xscale")
        _shape(Xq, (S, K), "Xq")
        _shape(xscale, (S,), "xscale")
        _same_device(X, positions=positions, Xq=Xq, xscale=xscale)
        _check(load_library().llmint8_quantize_rows(
            X.data_ptr(), _DTYPES[X.dtype], T, K, None if positions is None else positions.data_ptr(), copies, S,
            Xq.data_ptr(), xscale.data_ptr(), st), "llmint8_quantize_rows")
    return Xq, xscale


def _product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y, stream, where):
    grouped = offsets is not None
    nd = 3 if grouped else 2
    _need(Xq, torch.int8, 2, "Xq")
    _need(xscale, torch.float32, 1, "xscale")
    _need(Wq, torch.int8, nd, "Wq")
    _need(Wscale, torch.float32, nd - 1, "Wscale")
    S, K = Xq.shape
    N = Wq.shape[-2]
    lead = tuple(Wq.shape[:-2])
    _shape(Wq, lead + (N, K), "Wq")
    _shape(xscale, (S,), "xscale")
    _shape(Wscale, lead + (N,), "Wscale")
    if bias is not None:
        _need(bias, torch.float32, nd - 1, "bias")
        _shape(bias, lead + (N,), "bias")
    if grouped:
        _need(offsets, torch.int32, 1, "offsets")
        _shape(offsets, (lead[0] + 1,), "offsets")
    if gated and N % 32:
        raise ValueError(f"a gated product needs N = 2 F with F a multiple of 16, got N = {N}")
    No = N // 2 if gated else N
    if Y is not None:
        dtype = Y.dtype
    code = _out_dtype(dtype)
    _same_device(Xq, xscale=xscale, offsets=offsets, Wq=Wq, Wscale=Wscale, bias=bias, Y=Y)
    with _On(Xq.device, stream) as st:
        if Y is None:
            Y = torch.empty((S, No), dtype=dtype, device=Xq.device)
        else:
            _need(Y, dtype, 2, "Y")
            _shape(Y, (S, No), "Y")
        lib = load_library()
        b = None if bias is None else bias.data_ptr()
        if grouped:
            rc = lib.llmint8_grouped_matmul(Xq.data_ptr(), xscale.data_ptr(), S, K, offsets.data_ptr(), lead[0],
                                            Wq.data_ptr(), Wscale.data_ptr(), b, N, int(bool(gated)), Y.data_ptr(),
                                            code, st)
        else:
            rc = lib.llmint8_scaled_matmul(Xq.data_ptr(), xscale.data_ptr(), S, K, Wq.data_ptr(), Wscale.data_ptr(),
                                           b, N, int(bool(gated)), Y.data_ptr(), code, st)
        _check(rc, where)
    return Y


def llmint8_scaled_matmul(Xq: torch.Tensor, xscale: torch.Tensor, Wq: torch.Tensor, Wscale: torch.Tensor,
                          bias: torch.Tensor | None = None, gated: bool = False, dtype=torch.float16,
                          Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [T, N] = (Xq Wq^T) * xscale[:, None] * Wscale (+ bias) of int8 codes
    Xq [T, K], Wq [N, K] with float32 scales per token and per output channel.
    gated: N = 2 F (gate rows first), Y [T, F] = silu(gate) * value.  The output
    has `dtype`, or Y's."""
    return _product(Xq, xscale, None, Wq, Wscale, bias, gated, dtype, Y, stream, "llmint8_scaled_matmul")


def llmint8_grouped_matmul(Xq: torch.Tensor, xscale: torch.Tensor, offsets: torch.Tensor, Wq: torch.Tensor,
                           Wscale: torch.Tensor, bias: torch.Tensor | None = None, gated: bool = False,
                           dtype=torch.float16, Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """llmint8_scaled_matmul for rows grouped by expert: rows offsets[e] ..
    offsets[e + 1] - 1 of Xq [S, K] with Wq[e], Wscale[e], bias[e] of Wq
    [E, N, K], Wscale [E, N], bias [E, N]; offsets int32 [E + 1] on the device.
    Rows of Y outside the groups are left as they were."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a CUDA tensor")
    return _product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y, stream, "llmint8_grouped_matmul")


def llmint8_expert_positions(ids: torch.Tensor, experts: int, positions: torch.Tensor | None = None,
                             offsets: torch.Tensor | None = None, stream=None):
    """The order of a router's choices ids [T, k] (int32 or int64) by expert ->
    (positions int32 [T, k], offsets int32 [experts + 1]): expert e's rows are
    offsets[e] .. offsets[e + 1] - 1, stable in the order of ids; a choice
    outside [0, experts) has position -1."""
    if isinstance(ids, torch.Tensor) and ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    _need(ids, ids.dtype if isinstance(ids, torch.Tensor) else None, 2, "ids")
    T, k = ids.shape
    experts = int(experts)
    with _On(ids.device, stream) as st:
        positions = torch.empty((T, k), dtype=torch.int32, device=ids.device) if positions is None else positions
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device) if offsets is None else offsets
        _need(positions, torch.int32, 2, "positions")
        _need(offsets, torch.int32, 1, "offsets")
        _shape(positions, (T, k), "positions")
        _shape(offsets, (experts + 1,), "offsets")
        _same_device(ids, positions=positions, offsets=offsets)
        _check(load_library().llmint8_expert_positions(
            ids.data_ptr(), ids.element_size(), T, k, experts, positions.data_ptr(), offsets.data_ptr(), st),
            "llmint8_expert_positions")
    return positions, offsets


def llmint8_expert_combine(Y: torch.Tensor, positions: torch.Tensor, weights: torch.Tensor, dtype=None,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [T, N]: out[t] = sum_j weights[t, j] Y[positions[t, j]] over the
    positions >= 0 (Y [S, N], positions int32 [T, k], weights float32 [T, k]),
    in `dtype` (Y's by default, or out's)."""
    _float(Y, 2, "Y")
    _need(positions, torch.int32, 2, "positions")
    _need(weights, torch.float32, 2, "weights")
    S, N = Y.shape
    T, k = positions.shape
    _shape(weights, (T, k), "weights")
    dtype = out.dtype if out is not None else Y.dtype if dtype is None else dtype
    code = _out_dtype(dtype)
    _same_device(Y, positions=positions, weights=weights, out=out)
    with _On(Y.device, stream) as st:
        if out is None:
            out = torch.empty((T, N), dtype=dtype, device=Y.device)
        else:
            _need(out, dtype, 2, "out")
            _shape(out, (T, N), "out")
        _check(load_library().llmint8_expert_combine(
            Y.data_ptr(), _DTYPES[Y.dtype], S, N, positions.data_ptr(), weights.data_ptr(), T, k, out.data_ptr(),
            code, st), "llmint8_expert_combine")
    return out
