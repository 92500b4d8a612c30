"""Block-scaled 8-bit floats: quantisation, matrix product, weight gradient.

A matrix is held as codes (``torch.float8_e4m3fn`` or ``torch.float8_e5m2``)
and one fp32 scale for each block of 128 columns, per row ("rows": activations
and gradients) or per 128 rows ("tiles": weights); a value is code * scale.
The codes and scales of a layer's input serve twice: as the operand of the
forward product and as the 8-bit checkpoint that the backward pass reads.

Like the library's other ops, every op here writes into tensors that the
caller owns, enqueues its kernels on one stream and returns (the products:
the workspace, to be passed to the next call on that stream; one that is passed
and too small grows).  Tensors may have any non-negative strides.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _native

_FP8 = {torch.float8_e4m3fn: _native.IRIS_E4M3, torch.float8_e5m2: _native.IRIS_E5M2}
_DT = {torch.float16: _native.IRIS_F16, torch.bfloat16: _native.IRIS_BF16, torch.float32: _native.IRIS_F32}
_DT16 = {torch.float16: _native.IRIS_F16, torch.bfloat16: _native.IRIS_BF16}
_BLOCK = 128
_ROWS = {"rows": 1, "tiles": _BLOCK}


def _blocks(n: int) -> int:
    return (n + _BLOCK - 1) // _BLOCK


def _refuse(name: str, t, shape, dtypes, dims: int, index: int) -> None:
    """Say what is wrong with an argument that _lead, _mat or _vec did not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} is not a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has type {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, not {dims}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a CUDA device")
    if t.get_device() != index >= 0:
        raise ValueError(f"{name} is on {t.device}, not cuda:{index}")
    raise ValueError(f"{name} is not contiguous")


def _lead(name: str, t: torch.Tensor, dtypes):
    """(data, row stride, column stride), rows, columns and CUDA device of a
    call's first matrix, of one of these types."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == 2 and t.is_cuda):
        _refuse(name, t, None, dtypes, 2, -1)
    rows, cols = t.shape
    r, c = t.stride()
    return (t.data_ptr(), r, c), rows, cols, t.get_device()


def _mat(name: str, t: torch.Tensor, shape, dtypes, index: int):
    """(data, row stride, column stride) of a matrix of this shape and one of
    these types on CUDA device `index`."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.get_device() == index:
            r, c = t.stride()
            return t.data_ptr(), r, c
    except AttributeError:
        pass
    _refuse(name, t, shape, dtypes, 2, index)


def _vec(name: str, t: torch.Tensor, n: int, dtypes, index: int) -> int:
    """Address of a contiguous 1-D tensor of n elements."""
    try:
        if t.dtype in dtypes and t.shape == (n,) and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, (n,), dtypes, 1, index)


# Tells autograd that tensors were written by address: a backward pass that kept
# what was there before is an error then.
_written = torch._C._increment_version


def _cfgp(config):
    if config is None:
        return None
    if isinstance(config, str):
        if config != "auto":
            raise ValueError(f"unknown config {config!r}")
        return None  # the estimate from the sizes
    from . import make_config
    return ctypes.byref(make_config(**config) if isinstance(config, dict) else config)


def _stream(stream, index: int) -> int:
    if stream is None:
        # the raw handle; building a torch.cuda.Stream would cost as much as the launch
        return torch._C._cuda_getCurrentRawStream(index)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_F32 = (torch.float32,)


def empty_fp8(M: int, K: int, block: str = "rows", dtype: torch.dtype = torch.float8_e4m3fn, device="cuda"):
    """Uninitialised (codes, scales) for an M x K matrix: code rows on 16
    bytes, so that products read them in place, and "rows" scales with the
    rows next to each other in memory."""
    if block not in _ROWS:
        raise ValueError(f"unknown block {block!r}")
    if dtype not in _FP8:
        raise TypeError(f"{dtype} is not an 8-bit float type")
    codes = torch.empty(M, (K + 15) // 16 * 16, dtype=dtype, device=device)[:, :K]
    if block == "rows":
        return codes, torch.empty(_blocks(K), M, dtype=torch.float32, device=device).t()
    return codes, torch.empty(_blocks(M), _blocks(K), dtype=torch.float32, device=device)


def quantize_fp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, block: str = "rows",
                 pow2: bool = True, stream=None) -> None:
    """Quantise x (M, K) (f16, bf16 or f32) into codes (M, K) and scales:
    (M, ceil(K/128)) for "rows", (ceil(M/128), ceil(K/128)) for "tiles".

    With ``pow2`` a block's scale is the smallest power of two that takes its
    largest finite magnitude into the codes' range, and scaled codes are exact
    bf16 numbers (f16 numbers too for f16 input, but for 65536, to which codes
    round what is close to f16's largest); without it the scale maps that
    magnitude to the largest code.  NaN and infinities become the NaN code and leave the scale to the
    block's other elements; zero blocks get the smallest scale."""
    if block not in _ROWS:
        raise ValueError(f"unknown block {block!r}")
    mx, M, K, index = _lead("x", x, _DT)
    mc = _mat("codes", codes, (M, K), _FP8, index)
    ms = _mat("scales", scales, (M if block == "rows" else _blocks(M), _blocks(K)), _F32, index)
    args = _native.pack_quantize_fp8(*mx, *mc, *ms, M, K, _DT[x.dtype], _FP8[codes.dtype], _ROWS[block], bool(pow2))
    lib, st = _native.load(), _stream(stream, index)
    if index == torch._C._cuda_getDevice():
        rc = lib.iris_b200_quantize_fp8(args, st)
    else:
        with torch.cuda.device(index):
            rc = lib.iris_b200_quantize_fp8(args, st)
    if rc:
        _native.check("iris_b200_quantize_fp8", rc)
    _written((codes, scales))


def _need(name: str, args, cfg) -> int:
    """Bytes of workspace of a product."""
    size, n = "iris_b200_" + name + "_workspace_size", ctypes.c_size_t(0)
    _native.check(size, getattr(_native.load(), size)(args, cfg, ctypes.byref(n)))
    return int(n.value)


def _product(name: str, fn, args, out, config, ws, index: int, stream):
    """One product with the given workspace, grown where it is too small, or with a new one; `out` is marked as written."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _product(name, fn, args, out, config, ws, index, stream)
    cfg, st = _cfgp(config), _stream(stream, index)
    if ws is None:
        from . import _ws
        ws = _ws(None, _need(name, args, cfg), torch.device("cuda", index), stream)
    elif ws.buf.get_device() != index:
        raise ValueError(f"the workspace is on {ws.buf.device}, not cuda:{index}")
    # a product may be several launches: those of two threads must not mix
    with ws._lock:
        if ws._capture and ws._elsewhere(st):
            from . import _on
            with _on(stream, index):
                ws._grow(ws.nbytes)
        rc = fn(args, cfg, ws.buf.data_ptr(), ws.nbytes, st)
        if rc == _native.IRIS_ENOWS:
            from . import _on
            with _on(stream, index):
                ws._grow(_need(name, args, cfg))
            rc = fn(args, cfg, ws.buf.data_ptr(), ws.nbytes, st)
    if rc:
        _native.check("iris_b200_" + name, rc)
    if out is not None:
        _written((out,))
    return ws


def matmul_fp8(A: torch.Tensor, A_scale: torch.Tensor, B: torch.Tensor, B_scale: torch.Tensor, out: torch.Tensor,
               bias: Optional[torch.Tensor] = None, config=None, workspace=None, stream=None):
    """out = (A * A_scale) @ (B * B_scale) + bias.

    A (M, K) codes with "rows" scales (M, ceil(K/128)); B (K, N) codes with
    "tiles" scales (ceil(K/128), ceil(N/128)), in either order: the transpose
    of a quantised matrix is ``codes.t(), scales.t()``.  bias (N,) and out
    (M, N) are f16, bf16 or f32.  The 128-deep blocks are summed in fp32 and
    rounded once.  Returns the workspace."""
    ma, M, K, index = _lead("A", A, _FP8)
    mb, rows, N, b_index = _lead("B", B, _FP8)
    if b_index != index:
        _refuse("B", B, None, _FP8, 2, index)
    if rows != K:
        raise ValueError(f"A has {K} columns and B has {rows} rows")
    kb = _blocks(K)
    msa = _mat("A_scale", A_scale, (M, kb), _F32, index)
    msb = _mat("B_scale", B_scale, (kb, _blocks(N)), _F32, index)
    mo = _mat("out", out, (M, N), _DT, index)
    bias_ptr, bias_dt = 0, _native.IRIS_F32
    if bias is not None:
        bias_ptr, bias_dt = _vec("bias", bias, N, _DT, index), _DT[bias.dtype]
    args = _native.pack_matmul_fp8(*ma, *msa, *mb, *msb, *mo, bias_ptr, M, N, K, _FP8[A.dtype], _FP8[B.dtype], bias_dt,
                                   _DT[out.dtype])
    return _product("matmul_fp8", _native.load().iris_b200_matmul_fp8, args, out, config, workspace, index, stream)


def weight_grad_fp8(X: torch.Tensor, X_scale: torch.Tensor, dY: torch.Tensor, out: torch.Tensor, config=None,
                    workspace=None, stream=None):
    """out = (X * X_scale)^T @ dY: the weight gradient (K, N) of a linear layer
    from the 8-bit checkpoint of its input.

    X (M, K) codes with "rows" scales (M, ceil(K/128)); dY (M, N) f16 or bf16;
    out f16, bf16 or f32.  X's values enter in dY's type, exactly where the
    scales are powers of two; for f16, values past its range or below its
    finest step are held times a power of two for each run of 512 tokens, and
    lose at most what lies under 2^-39 of the largest value that the run's
    scales allow.  Returns the workspace."""
    mx, M, K, index = _lead("X", X, _FP8)
    md, rows, N, dy_index = _lead("dY", dY, _DT16)
    if dy_index != index:
        _refuse("dY", dY, None, _DT16, 2, index)
    if rows != M:
        raise ValueError(f"X has {M} rows and dY has {rows}")
    ms = _mat("X_scale", X_scale, (M, _blocks(K)), _F32, index)
    mo = _mat("out", out, (K, N), _DT, index)
    args = _native.pack_weight_grad_fp8(*mx, *ms, *md, *mo, M, N, K, _FP8[X.dtype], _DT[dY.dtype], _DT[out.dtype], 0)
    return _product("weight_grad_fp8", _native.load().iris_b200_weight_grad_fp8, args, out, config, workspace, index, stream)


_layer_workspaces = {}  # by device and stream


def fp8_workspace(device="cuda"):
    """The workspace of ``fp8_linear`` calls on the device's current stream that
    are given none: one per stream, kept and grown as needed.  Errors on the
    device in such calls are found by ``query_status(fp8_workspace())``."""
    from . import Workspace
    index = torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    key = index, _stream(None, index)
    ws = _layer_workspaces.get(key)
    if ws is None:
        ws = _layer_workspaces.setdefault(key, Workspace(256, torch.device("cuda", index), wait=False))
    return ws


def _layer_workspace(workspace, device):
    """The caller's; else the stream's; else, in a capture, whose graph may run
    beside that stream's work, a new one."""
    if workspace is not None:
        return workspace
    if torch.cuda.is_current_stream_capturing():
        from . import Workspace
        return Workspace(256, device, wait=False)
    index = device.index
    return _layer_workspaces.get((index, torch._C._cuda_getCurrentRawStream(index))) or fp8_workspace(device)


class _Fp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, W_scale, weight, bias, grad_dtype, workspace):
        x2 = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])  # sizes of zero among them
        M, K = x2.shape
        codes, scales = empty_fp8(M, K, "rows", device=x.device)
        quantize_fp8(x2, codes, scales)
        y = torch.empty(M, W.shape[1], dtype=x.dtype, device=x.device)
        matmul_fp8(codes, scales, W, W_scale, y, bias=bias, workspace=_layer_workspace(workspace, x.device))
        # the 8-bit checkpoint is all that is kept of x
        ctx.save_for_backward(codes, scales, W, W_scale)
        ctx.x_shape, ctx.grad_dtype, ctx.workspace = x.shape, grad_dtype, workspace
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y.reshape(*x.shape[:-1], W.shape[1])

    # the kernels' gradients have no derivatives of their own: asking for second
    # ones is an error, not a sum without some of its terms
    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        codes, scales, W, W_scale = ctx.saved_tensors
        M, K = codes.shape
        N = W.shape[1]
        dy2 = dy.reshape(M, N)
        dx = dw = db = None
        ws = _layer_workspace(ctx.workspace, dy.device)
        if ctx.needs_input_grad[0]:
            dcodes, dscales = empty_fp8(M, N, "rows", ctx.grad_dtype, dy.device)
            quantize_fp8(dy2, dcodes, dscales)
            dx = torch.empty(M, K, dtype=dy.dtype, device=dy.device)
            matmul_fp8(dcodes, dscales, W.t(), W_scale.t(), dx, workspace=ws)
            dx = dx.reshape(ctx.x_shape)
        if ctx.needs_input_grad[3]:
            dw = torch.empty(K, N, dtype=torch.float32, device=dy.device)
            weight_grad_fp8(codes, scales, dy2, dw, workspace=ws)
        if ctx.bias_dtype is not None and ctx.needs_input_grad[4]:
            db = dy2.sum(0, dtype=torch.float32).to(ctx.bias_dtype)
        return dx, None, None, dw, db, None, None


def fp8_linear(x: torch.Tensor, W: torch.Tensor, W_scale: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, grad_dtype: torch.dtype = torch.float8_e5m2, workspace=None):
    """Differentiable y = x @ (W * W_scale) + bias, x (..., K) f16 or bf16.

    W (K, N) codes with "tiles" scales; ``weight`` is the fp32 master weight
    (K, N) that W was quantised from and that receives the gradient (None: no
    weight gradient).  The forward pass quantises x once; codes and scales are
    the product's operand and, in place of x, what is kept for the backward
    pass: dx = quantised(dy) @ W^T, dweight = checkpoint^T @ dy.

    All products use ``workspace``, which grows to what they need and reports
    their device errors to ``query_status``; without one they use the stream's,
    ``fp8_workspace()``.  In a graph capture, where that belongs to work beside
    the graph, calls without one make their own: pass one to be told of errors."""
    if x.dim() < 1 or x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x is a f16 or bf16 tensor (..., K)")
    if weight is not None and (weight.dtype != torch.float32 or weight.shape != W.shape):
        raise ValueError(f"weight is a float32 tensor of shape {tuple(W.shape)}")
    return _Fp8Linear.apply(x, W, W_scale, weight, bias, grad_dtype, workspace)
