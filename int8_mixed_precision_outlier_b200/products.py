"""Python binding of the int8 products with token and channel scales, dense and
grouped by expert, and of the row quantisation, expert positions and combine
that go with them (include/llmint8.h).

Argument marshalling only, as llmint8.py: dtypes, shapes, devices and layouts
are checked, outputs that are not given are allocated on the call's stream, and
the library's kernels do the rest.  Calls run on the device of their tensors,
whichever is current.  For few tokens the host's time is what a call costs, so
each operand is checked by one test of all its properties, which is taken apart
only to name what is wrong.
"""
from __future__ import annotations

import torch

from . import llmint8 as _base
from .llmint8 import _check, _need

_F16, _BF16, _F32 = torch.float16, torch.bfloat16, torch.float32
_I8, _I32, _I64 = torch.int8, torch.int32, torch.int64
_DTYPES = {_F16: 0, _BF16: 1, _F32: 2}
MAX_EXPERTS = 1024

_Tensor = torch.Tensor
# _C._cuda_getCurrentRawStream and _cuda_getDevice give the stream's pointer and
# the device's index alone, 3 us less than by way of a Stream object.  A torch
# without CUDA has neither, so they are looked up in a call.
_C = torch._C


def _lib():
    return _base._LIB or _base.load_library()


def _refuse(t, dtype, shape, name, index):
    """Raises for what is wrong with an operand (see _operand)."""
    _need(t, dtype, len(shape), name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _operand(t, dtype, shape, name, index):
    """A contiguous CUDA tensor of this type and shape on device `index`."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _refuse(t, dtype, shape, name, index)


def _first(t, dtypes, ndim, name) -> int:
    """The device of a call's first operand; `dtypes` None: any of the float types."""
    if isinstance(t, _Tensor) and dtypes is None and t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    if isinstance(t, _Tensor) and dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, got {t.dtype}")
    if not (isinstance(t, _Tensor) and t.is_cuda and t.dim() == ndim and t.is_contiguous()):
        _need(t, t.dtype if isinstance(t, _Tensor) else None, ndim, name)
    return t.get_device()


def _out_dtype(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
    return code


def _run(index: int, stream, call):
    """call(pointer of the stream) with the tensors' device and the call's
    stream current, so that an output belongs to the stream that writes it."""
    if stream is None:
        if index == _C._cuda_getDevice():
            return call(_C._cuda_getCurrentRawStream(index))
        with torch.cuda.device(index):
            return call(_C._cuda_getCurrentRawStream(index))
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def llmint8_quantize_rows(X: torch.Tensor, positions: torch.Tensor | None = None, Xq: torch.Tensor | None = None,
                          xscale: torch.Tensor | None = None, stream=None):
    """X [T, K] (float16, bfloat16 or float32) -> (Xq int8, xscale float32), one
    scale per row: max|x| / 127.

    With positions (int32 [T, k], llmint8_expert_positions) row t is written to
    every row positions[t, j] >= 0 of Xq [S, K] and xscale [S]; S is T k unless
    Xq is given, and rows that no position names are left as they were.
    Positions must be distinct: what a row that is named twice holds is not
    defined, not even that its codes and scale are of one token.  A row with a NaN or an infinity gets the scale
    NaN and codes 0."""
    try:
        T, K = X.shape
        S = T
        if positions is not None:
            copies = positions.shape[1]
            S = T * copies if Xq is None else Xq.shape[0]
        index = X.get_device()
        # _check_quantize in one expression
        fine = (index >= 0 and X.dtype in _DTYPES and X.is_contiguous()
                and (positions is None or copies > 0 and positions.dtype is _I32 and positions.shape == (T, copies)
                     and positions.is_contiguous() and positions.get_device() == index)
                and (Xq is None or Xq.dtype is _I8 and Xq.shape == (S, K) and Xq.is_contiguous()
                     and Xq.get_device() == index)
                and (xscale is None or xscale.dtype is _F32 and xscale.shape == (S,) and xscale.is_contiguous()
                     and xscale.get_device() == index))
    except (AttributeError, ValueError, IndexError):
        fine = False
    if not fine:
        _check_quantize(X, positions, Xq, xscale)
    if stream is not None or index != _C._cuda_getDevice():
        return _run(index, stream, lambda st: _launch_quantize(X, positions, Xq, xscale, S, st))
    return _launch_quantize(X, positions, Xq, xscale, S, _C._cuda_getCurrentRawStream(index))


def _check_quantize(X, positions, Xq, xscale):
    """Raises for what is wrong with llmint8_quantize_rows' arguments, one by one."""
    index = _first(X, None, 2, "X")
    T, K = X.shape
    S = T
    if positions is not None:
        _first(positions, (_I32,), 2, "positions")
        _operand(positions, _I32, (T, positions.shape[1]), "positions", index)
        if positions.shape[1] < 1:
            raise ValueError("positions must have a column")
        S = positions.numel()
        if Xq is not None:
            _first(Xq, (_I8,), 2, "Xq")
            S = Xq.shape[0]
    if Xq is not None:
        _operand(Xq, _I8, (S, K), "Xq", index)
    if xscale is not None:
        _operand(xscale, _F32, (S,), "xscale", index)


def _launch_quantize(X, positions, Xq, xscale, S, st):
    T, K = X.shape
    if Xq is None:
        Xq = torch.empty(S, K, dtype=_I8, device=X.device)
    if xscale is None:
        xscale = torch.empty(S, dtype=_F32, device=X.device)
    at, copies = (None, 0) if positions is None else (positions.data_ptr(), positions.shape[1])
    rc = _lib().llmint8_quantize_rows(X.data_ptr(), _DTYPES[X.dtype], T, K, at, copies, S, Xq.data_ptr(),
                                      xscale.data_ptr(), st)
    if rc:
        _check(rc, "llmint8_quantize_rows")
    return Xq, xscale


def _check_product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y):
    """Raises for what is wrong with a product's arguments, one by one."""
    index = _first(Xq, (_I8,), 2, "Xq")
    _first(Wq, (_I8,), 2 if offsets is None else 3, "Wq")
    S, K = Xq.shape
    rows = tuple(Wq.shape[:-1])
    _operand(Wq, _I8, rows + (K,), "Wq", index)
    _operand(xscale, _F32, (S,), "xscale", index)
    _operand(Wscale, _F32, rows, "Wscale", index)
    if bias is not None:
        _operand(bias, _F32, rows, "bias", index)
    if offsets is not None:
        _operand(offsets, _I32, (rows[0] + 1,), "offsets", index)
    if gated and rows[-1] % 32:
        raise ValueError(f"a gated product needs N = 2 F with F a multiple of 16, got N = {rows[-1]}")
    _out_dtype(dtype if Y is None else Y.dtype)
    if Y is not None:
        _operand(Y, Y.dtype, (S, rows[-1] // 2 if gated else rows[-1]), "Y", index)


def _product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y, stream, where):
    try:
        S, K = Xq.shape
        shape = Wq.shape
        rows = shape[:-1]
        N = No = rows[-1]
        if gated:
            No = N // 2
        if Y is not None:
            dtype = Y.dtype
        index = Xq.get_device()
        # _check_product in one expression
        fine = (index >= 0 and shape[-1] == K and Xq.dtype is _I8 and Wq.dtype is _I8 and xscale.dtype is _F32
                and Wscale.dtype is _F32 and xscale.shape == (S,) and Wscale.shape == rows and Xq.is_contiguous()
                and Wq.is_contiguous() and xscale.is_contiguous() and Wscale.is_contiguous()
                and Wq.get_device() == index and xscale.get_device() == index and Wscale.get_device() == index
                and (len(rows) == 1 if offsets is None else len(rows) == 2 and offsets.dtype is _I32
                     and offsets.shape == (rows[0] + 1,) and offsets.is_contiguous() and offsets.get_device() == index)
                and (bias is None or bias.dtype is _F32 and bias.shape == rows and bias.is_contiguous()
                     and bias.get_device() == index)
                and (Y is None or Y.shape == (S, No) and Y.is_contiguous() and Y.get_device() == index)
                and (not gated or N % 32 == 0) and dtype in _DTYPES)
    except (AttributeError, ValueError, IndexError):
        fine = False
    if not fine:
        _check_product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y)
    if stream is not None or index != _C._cuda_getDevice():
        return _run(index, stream,
                    lambda st: _launch_product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y, st, where))
    return _launch_product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y,
                           _C._cuda_getCurrentRawStream(index), where)


def _launch_product(Xq, xscale, offsets, Wq, Wscale, bias, gated, dtype, Y, st, where):
    S, K = Xq.shape
    N = Wq.shape[-2]
    if Y is None:
        Y = torch.empty(S, N // 2 if gated else N, dtype=dtype, device=Xq.device)
    b = None if bias is None else bias.data_ptr()
    lib = _lib()
    if offsets is None:
        rc = lib.llmint8_scaled_matmul(Xq.data_ptr(), xscale.data_ptr(), S, K, Wq.data_ptr(), Wscale.data_ptr(), b, N,
                                       1 if gated else 0, Y.data_ptr(), _DTYPES[dtype], st)
    else:
        rc = lib.llmint8_grouped_matmul(Xq.data_ptr(), xscale.data_ptr(), S, K, offsets.data_ptr(), Wq.shape[0],
                                        Wq.data_ptr(), Wscale.data_ptr(), b, N, 1 if gated else 0, Y.data_ptr(),
                                        _DTYPES[dtype], st)
    if rc:
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
    try:
        T, k = ids.shape
        index = ids.get_device()
        # _check_positions in one expression
        fine = (index >= 0 and (ids.dtype is _I64 or ids.dtype is _I32) and ids.is_contiguous()
                and 0 < experts <= MAX_EXPERTS
                and (positions is None or positions.dtype is _I32 and positions.shape == (T, k)
                     and positions.is_contiguous() and positions.get_device() == index)
                and (offsets is None or offsets.dtype is _I32 and offsets.shape == (experts + 1,)
                     and offsets.is_contiguous() and offsets.get_device() == index))
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _check_positions(ids, experts, positions, offsets)
    if stream is not None or index != _C._cuda_getDevice():
        return _run(index, stream, lambda st: _launch_positions(ids, experts, positions, offsets, st))
    return _launch_positions(ids, experts, positions, offsets, _C._cuda_getCurrentRawStream(index))


def _check_positions(ids, experts, positions, offsets):
    """Raises for what is wrong with llmint8_expert_positions' arguments, one by one."""
    index = _first(ids, (_I32, _I64), 2, "ids")
    if experts < 1 or experts > MAX_EXPERTS:
        raise ValueError(f"experts must be in [1, {MAX_EXPERTS}], got {experts}")
    if positions is not None:
        _operand(positions, _I32, tuple(ids.shape), "positions", index)
    if offsets is not None:
        _operand(offsets, _I32, (experts + 1,), "offsets", index)


def _launch_positions(ids, experts, positions, offsets, st):
    T, k = ids.shape
    if positions is None:
        positions = torch.empty(T, k, dtype=_I32, device=ids.device)
    if offsets is None:
        offsets = torch.empty(experts + 1, dtype=_I32, device=ids.device)
    rc = _lib().llmint8_expert_positions(ids.data_ptr(), 8 if ids.dtype is _I64 else 4, T, k, experts,
                                         positions.data_ptr(), offsets.data_ptr(), st)
    if rc:
        _check(rc, "llmint8_expert_positions")
    return positions, offsets


def llmint8_expert_combine(Y: torch.Tensor, positions: torch.Tensor, weights: torch.Tensor, dtype=None,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [T, N]: out[t] = sum_j weights[t, j] Y[positions[t, j]] over the
    positions >= 0 (Y [S, N], positions int32 [T, k], weights float32 [T, k]),
    in `dtype` (Y's by default, or out's)."""
    try:
        N = Y.shape[1]
        shape = positions.shape
        T, k = shape
        dtype = out.dtype if out is not None else Y.dtype if dtype is None else dtype
        index = Y.get_device()
        # _check_combine in one expression
        fine = (index >= 0 and Y.dtype in _DTYPES and dtype in _DTYPES and Y.ndim == 2 and Y.is_contiguous()
                and positions.dtype is _I32 and positions.is_contiguous() and positions.get_device() == index
                and weights.dtype is _F32 and weights.shape == shape and weights.is_contiguous()
                and weights.get_device() == index
                and (out is None or out.shape == (T, N) and out.is_contiguous() and out.get_device() == index))
    except (AttributeError, ValueError, IndexError):
        fine = False
    if not fine:
        _check_combine(Y, positions, weights, dtype, out)
    if stream is not None or index != _C._cuda_getDevice():
        return _run(index, stream, lambda st: _launch_combine(Y, positions, weights, dtype, out, st))
    return _launch_combine(Y, positions, weights, dtype, out, _C._cuda_getCurrentRawStream(index))


def _check_combine(Y, positions, weights, dtype, out):
    """Raises for what is wrong with llmint8_expert_combine's arguments, one by one."""
    index = _first(Y, None, 2, "Y")
    _first(positions, (_I32,), 2, "positions")
    shape = tuple(positions.shape)
    _operand(positions, _I32, shape, "positions", index)
    _operand(weights, _F32, shape, "weights", index)
    _out_dtype(out.dtype if out is not None else Y.dtype if dtype is None else dtype)
    if out is not None:
        _operand(out, out.dtype, (shape[0], Y.shape[1]), "out", index)


def _launch_combine(Y, positions, weights, dtype, out, st):
    S, N = Y.shape
    T, k = positions.shape
    if out is None:
        out = torch.empty(T, N, dtype=dtype, device=Y.device)
    rc = _lib().llmint8_expert_combine(Y.data_ptr(), _DTYPES[Y.dtype], S, N, positions.data_ptr(),
                                       weights.data_ptr(), T, k, out.data_ptr(), _DTYPES[dtype], st)
    if rc:
        _check(rc, "llmint8_expert_combine")
    return out


class Int8Experts:
    """A mixture of gated experts with int8 weights:

        y[t] = sum_j weights[t, j] W2[e] (silu(G[e] x[t]) * (V[e] x[t])),  e = ids[t, j],  W1[e] = [G[e]; V[e]]

    W1 [E, 2 F, K] and W2 [E, N, F] (float16, bfloat16 or float32, K and F
    multiples of 16) are quantised once, per output channel; activations per
    row, before each product.  A call takes X [T, K], a router's ids [T, k]
    (int32 or int64; outside [0, E): no expert) and weights [T, k] (float32)
    and returns [T, N] in X's type.  The hidden rows stay in float32 until they
    are quantised: rounding them to 16 bits first would move their codes.  The
    experts' outputs are rounded to X's type before the weighted sum, which
    halves what the combine reads and costs one rounding per term.  Buffers are
    allocated by each call on its stream, so calls on several streams and
    captured graphs do not meet.
    """

    def __init__(self, W1: torch.Tensor, W2: torch.Tensor):
        if W1.dim() != 3 or W2.dim() != 3 or W1.shape[0] != W2.shape[0] or W1.shape[1] != 2 * W2.shape[2]:
            raise ValueError(f"W1 must be [E, 2 F, K] and W2 [E, N, F], got {tuple(W1.shape)} and {tuple(W2.shape)}")
        self.E, two_f, self.K = W1.shape
        self.N, self.F = W2.shape[1:]
        if not 1 <= self.E <= MAX_EXPERTS:
            raise ValueError(f"experts must be in [1, {MAX_EXPERTS}], got {self.E}")
        if self.K % 16 or self.F % 16:
            raise ValueError(f"K and F must be multiples of 16, got {self.K} and {self.F}")
        q, s = llmint8_quantize_rows(W1.reshape(-1, self.K).contiguous())
        self.W1q, self.W1scale = q.view(self.E, two_f, self.K), s.view(self.E, two_f)
        q, s = llmint8_quantize_rows(W2.reshape(-1, self.F).contiguous())
        self.W2q, self.W2scale = q.view(self.E, self.N, self.F), s.view(self.E, self.N)

    def resident_weight_bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.W1q, self.W1scale, self.W2q, self.W2scale))

    def __call__(self, X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, stream=None) -> torch.Tensor:
        positions, offsets = llmint8_expert_positions(ids, self.E, stream=stream)
        Xq, xscale = llmint8_quantize_rows(X, positions, stream=stream)
        H = llmint8_grouped_matmul(Xq, xscale, offsets, self.W1q, self.W1scale, gated=True, dtype=_F32, stream=stream)
        Hq, hscale = llmint8_quantize_rows(H, stream=stream)
        Y = llmint8_grouped_matmul(Hq, hscale, offsets, self.W2q, self.W2scale, dtype=X.dtype, stream=stream)
        return llmint8_expert_combine(Y, positions, weights, stream=stream)
