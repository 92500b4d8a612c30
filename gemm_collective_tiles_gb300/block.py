"""The sides of a block's linear layers: a product with its epilogue, dropout,
the norms around a block's end.

As the library's other ops, ``matmul_act``, ``act_grad``, ``dropout_add``,
``norm_join`` and ``norm_join_grad`` write into tensors that the caller owns,
enqueue their kernels on one stream and return (those with a workspace: the
workspace, to be passed to the next call on that stream; one that is passed and
too small grows).  Tensors may have any non-negative strides; rows that start on
16 bytes are read and written fastest.  ``linear_act``, ``dropout`` and
``block_norm`` are the differentiable forms, which make their outputs; their
products and sums use the stream's workspace (``fp8_workspace``) where they are
given none.

Dropout takes its random bits from ``rng``, an int64 tensor (seed, offset) on
the device, and from an element's row and column (Philox4x32-10, 16 bits an
element: p is rounded to a multiple of 2^-16).  The same rng gives the same mask
in every op, forward and backward, so no mask is stored; a program adds 1 to the
offset, or to the seed, for each layer and step, by a kernel where it replays a
graph.
"""
from __future__ import annotations

import math
from typing import Optional

import torch
from torch.autograd import forward_ad

from . import _native
from .fp8 import (_DT, _DT16, _F32, _lead, _layer_workspace, _mat, _product, _refuse, _stream, _vec, _written)

_ACTS = {None: _native.IRIS_ACT_NONE, "relu": _native.IRIS_ACT_RELU, "gelu": _native.IRIS_ACT_GELU,
         "gelu_tanh": _native.IRIS_ACT_GELU_TANH, "silu": _native.IRIS_ACT_SILU}
_NORMS = {None: _native.IRIS_NORM_NONE, "rms": _native.IRIS_NORM_RMS, "layer": _native.IRIS_NORM_LAYER}
_NO_MAT = (0, 0, 0)
_I64 = (torch.int64,)


def _choice(name: str, value, table):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"unknown {name} {value!r}") from None


def _rng(p: float, rng, index: int) -> int:
    """Address of the random state that a dropout of p needs, or 0."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p is {p}, not between 0 and 1")
    if rng is None:
        if round(p * 65536) > 0:
            raise ValueError("dropout needs rng, an int64 tensor (seed, offset)")
        return 0
    return _vec("rng", rng, 2, _I64, index)


def _like(name: str, t, shape, dtype, index: int):
    """An optional matrix of this shape and type."""
    return _NO_MAT if t is None else _mat(name, t, shape, (dtype,), index)


def _run(name: str, args, index: int, stream) -> None:
    """A call without a workspace."""
    fn, st = getattr(_native.load(), "iris_b200_" + name), _stream(stream, index)
    if index == torch._C._cuda_getDevice():
        rc = fn(args, st)
    else:
        with torch.cuda.device(index):
            rc = fn(args, st)
    if rc:
        _native.check("iris_b200_" + name, rc)


def matmul_act(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor, bias: Optional[torch.Tensor] = None,
               act: Optional[str] = None, residual: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
               p: float = 0.0, rng: Optional[torch.Tensor] = None, config=None, workspace=None, stream=None):
    """z = A @ B + bias, out = residual + dropout(act(z)).

    A (M, K) and B (K, N) f16 or bf16, either order of each (a transposed view
    is read as it is); out (M, N) f16, bf16 or f32; bias (N,) any of the three;
    act None, "relu", "gelu" (by the normal distribution), "gelu_tanh" or
    "silu"; residual as out, out itself among them (which adds to out: a
    gradient buffer); z as out, None: not wanted.  Everything after the product
    is fp32, rounded once.  Returns the workspace."""
    a = _choice("activation", act, _ACTS)
    ma, M, K, index = _lead("A", A, _DT16)
    mb, rows, N, b_index = _lead("B", B, (A.dtype,))
    if b_index != index:
        _refuse("B", B, None, (A.dtype,), 2, index)
    if rows != K:
        raise ValueError(f"A has {K} columns and B has {rows} rows")
    mo = _mat("out", out, (M, N), _DT, index)
    mr = _like("residual", residual, (M, N), out.dtype, index)
    mz = _like("z", z, (M, N), out.dtype, index)
    bias_ptr, bias_dt = 0, 0
    if bias is not None:
        bias_ptr, bias_dt = _vec("bias", bias, N, _DT, index), _DT[bias.dtype]
    args = _native.pack_matmul_act(*ma, *mb, *mo, *mr, *mz, bias_ptr, _rng(p, rng, index), M, N, K, p, _DT[A.dtype],
                                   _DT[out.dtype], bias_dt, a)
    ws = _product("matmul_act", _native.load().iris_b200_matmul_act, args, out, config, workspace, index, stream)
    if z is not None:
        _written((z,))
    return ws


def act_grad(dy: torch.Tensor, z: Optional[torch.Tensor], dz: Optional[torch.Tensor], dbias: Optional[torch.Tensor] = None,
             act: Optional[str] = None, p: float = 0.0, rng: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """dz = dropout(dy) act'(z), dbias = the column sums of dz.

    dy (M, N) f16, bf16 or f32; z as dy (None without an activation); dz (M, N)
    and dbias (N,) of any of the three types, either None.  dz may be dy or z.
    Sums are fp32, of values before their rounding, in a fixed order.  Returns
    the workspace."""
    a = _choice("activation", act, _ACTS)
    md, M, N, index = _lead("dy", dy, _DT)
    if a and z is None:
        raise ValueError("the gradient of an activation needs z")
    mz = _like("z", z, (M, N), dy.dtype, index) if a else _NO_MAT
    mo, dz_dt = _NO_MAT, 0
    if dz is not None:
        mo, dz_dt = _mat("dz", dz, (M, N), _DT, index), _DT[dz.dtype]
    bias_ptr, bias_dt = 0, 0
    if dbias is not None:
        bias_ptr, bias_dt = _vec("dbias", dbias, N, _DT, index), _DT[dbias.dtype]
    args = _native.pack_act_grad(*md, *mz, *mo, bias_ptr, _rng(p, rng, index), M, N, p, _DT[dy.dtype], dz_dt, bias_dt, a)
    return _sums("act_grad", args, [t for t in (dz, dbias) if t is not None], workspace, index, stream)


def linear_act_grad(dy: torch.Tensor, x: Optional[torch.Tensor], weight: Optional[torch.Tensor], z: Optional[torch.Tensor],
                    dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                    dbias: Optional[torch.Tensor] = None, act: Optional[str] = None, p: float = 0.0,
                    rng: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """The gradients of residual + dropout(act(x @ weight + bias)) in one call:
    dz = dropout(dy) act'(z), dx = dz @ weight^T, dweight = x^T @ dz, dbias = the
    column sums of dz.

    dy (M, N), x (M, K), weight (K, N), z (M, N) (None without an activation), dx
    and dweight f16 or bf16, the same type; dbias (N,) f16, bf16 or f32.  Each of
    the three gradients may be None, and x or weight with the one that reads it.
    dz is rounded to that type, for the products, and lies in the workspace, which
    is returned."""
    a = _choice("activation", act, _ACTS)
    md, M, N, index = _lead("dy", dy, _DT16)
    types = (dy.dtype,)
    if a and z is None:
        raise ValueError("the gradient of an activation needs z")
    mz = _mat("z", z, (M, N), types, index) if a else _NO_MAT
    K = 0
    mx = mw = mdx = mdw = _NO_MAT
    if dx is not None:
        mw, K, _, _ = _lead("weight", weight, types)
        mw = _mat("weight", weight, (K, N), types, index)
        mdx = _mat("dx", dx, (M, K), types, index)
    if dweight is not None:
        mx, _, k, _ = _lead("x", x, types)
        if dx is not None and k != K:
            raise ValueError(f"x has {k} columns and weight has {K} rows")
        K = k
        mx = _mat("x", x, (M, K), types, index)
        mdw = _mat("dweight", dweight, (K, N), types, index)
    bias_ptr, bias_dt = 0, 0
    if dbias is not None:
        bias_ptr, bias_dt = _vec("dbias", dbias, N, _DT, index), _DT[dbias.dtype]
    args = _native.pack_linear_act_grad(*md, *mx, *mw, *mz, *mdx, *mdw, bias_ptr, _rng(p, rng, index), M, N, K, p,
                                        _DT[dy.dtype], bias_dt, a, 0)
    return _sums("linear_act_grad", args, [t for t in (dx, dweight, dbias) if t is not None], workspace, index, stream)


def _sums(name: str, args, outs, workspace, index: int, stream):
    """A call whose workspace holds sums over rows."""
    ws = _product(name, getattr(_native.load(), "iris_b200_" + name), args, outs[0], None, workspace, index, stream) \
        if outs else workspace
    if len(outs) > 1:
        _written(tuple(outs[1:]))
    return ws


def dropout_add(x: torch.Tensor, out: torch.Tensor, p: float, rng: Optional[torch.Tensor],
                residual: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = residual + dropout(x), (M, N) of one type, f16, bf16 or f32; out may
    be x or residual itself.  The gradient of x is the same call on out's."""
    mx, M, N, index = _lead("x", x, _DT)
    mo = _mat("out", out, (M, N), (x.dtype,), index)
    mr = _like("residual", residual, (M, N), x.dtype, index)
    _run("dropout", _native.pack_dropout(*mx, *mr, *mo, _rng(p, rng, index), M, N, p, _DT[x.dtype], 0), index, stream)
    _written((out,))


def _norm_vec(name: str, t, kind: int, D: int, index: int):
    """(address, type) of an optional vector of a norm."""
    if t is None:
        return 0, 0
    if not kind:
        raise ValueError(f"{name} without its norm")
    return _vec(name, t, D, _DT, index), _DT[t.dtype]


def _norm_args(y, h, n, x, gate, scale, post, post_weight, post_bias, pre, weight, bias, eps, stats):
    """The packed arguments of norm_join, as a tuple, and the device."""
    kind_post, kind_pre = _choice("norm", post, _NORMS), _choice("norm", pre, _NORMS)
    my, M, D, index = _lead("y", y, _DT)
    mx = mh = mg = _NO_MAT
    x_type, y_type = y.dtype, (y.dtype,)
    if x is not None:
        mx = _mat("x", x, (M, D), (x_type, torch.float32), index)
        x_type = x.dtype
    if h is not None:
        mh = _mat("h", h, (M, D), (x_type, torch.float32) if x is None else (x_type,), index)
        x_type = h.dtype
    gate_rows = gate_dt = 0
    if gate is not None:
        mg, gate_rows, cols, g_index = _lead("gate", gate, _DT)
        if g_index != index or cols != D:
            _refuse("gate", gate, (gate_rows, D), _DT, 2, index)
        if gate_rows < (M > 0) or gate_rows > max(M, 1) or gate_rows and M % gate_rows:
            raise ValueError(f"gate has {gate_rows} rows, which do not divide y's {M}")
        gate_dt = _DT[gate.dtype]
    mn = _NO_MAT if n is None else _mat("n", n, (M, D), y_type, index)
    pw, pw_dt = _norm_vec("post_weight", post_weight, kind_post, D, index)
    pb, pb_dt = _norm_vec("post_bias", post_bias, kind_post, D, index)
    w, w_dt = _norm_vec("weight", weight, kind_pre, D, index)
    b, b_dt = _norm_vec("bias", bias, kind_pre, D, index)
    st = 0
    if stats is not None:
        st = _mat("stats", stats, (M, 4), _F32, index)[0]
        if not stats.is_contiguous():
            raise ValueError("stats is not contiguous")
    return (*my, *mx, *mg, *mh, *mn, pw, pb, w, b, st, M, D, gate_rows, scale, eps, _DT[y.dtype], _DT[x_type], gate_dt, pw_dt, pb_dt,
            w_dt, b_dt, kind_post, kind_pre, 0), M, D, index, x_type


def norm_join(y: torch.Tensor, h: Optional[torch.Tensor], n: Optional[torch.Tensor], x: Optional[torch.Tensor] = None,
              gate: Optional[torch.Tensor] = None, scale: float = 1.0, post: Optional[str] = None,
              post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None, pre: Optional[str] = None,
              weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, eps: float = 1e-6,
              stats: Optional[torch.Tensor] = None, stream=None) -> None:
    """The end of a block and the start of the next: u = post-norm of y (or y),
    h = x + scale * gate * u, n = pre-norm of h.

    y (M, D) f16, bf16 or f32, n as y; x and h (M, D) of y's type or f32 (the
    residual stream), x None: not added; gate (G, D), each row for M / G rows of y:
    a learned scale (1, D), one per sequence, one per token (M, D), which may be no
    rows where M is 0; post, pre: None,
    "rms" or "layer", with optional weights and biases (D,); any of the three types
    for gate and vectors.  h None: not wanted; n None just where pre is.  stats
    (M, 4) f32, where given, takes what ``norm_join_grad`` needs.  h may be x
    itself, n may be y."""
    if (pre is None) != (n is None):
        raise ValueError("n is written by the pre-norm: both or neither")
    _norm_join(y, h, n, x, gate, scale, post, post_weight, post_bias, pre, weight, bias, eps, stats, stream)
    _written(tuple(t for t in (h, n, stats) if t is not None))


def _norm_join(y, h, n, x, gate, scale, post, post_weight, post_bias, pre, weight, bias, eps, stats, stream=None):
    """The call, and its arguments."""
    args, _, _, index, _ = _norm_args(y, h, n, x, gate, scale, post, post_weight, post_bias, pre, weight, bias, eps, stats)
    _run("norm_join", _native.pack_norm_join(*args), index, stream)
    return args


def norm_join_grad(y: torch.Tensor, stats: torch.Tensor, dh: Optional[torch.Tensor], dn: Optional[torch.Tensor],
                   x: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                   post: Optional[str] = None, post_weight: Optional[torch.Tensor] = None,
                   post_bias: Optional[torch.Tensor] = None, pre: Optional[str] = None, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-6, dy: Optional[torch.Tensor] = None,
                   dx: Optional[torch.Tensor] = None, dgate: Optional[torch.Tensor] = None,
                   dpost_weight: Optional[torch.Tensor] = None, dpost_bias: Optional[torch.Tensor] = None,
                   dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """The gradients of ``norm_join`` from those of h and n (either None): dy, dx,
    dgate and those of the vectors, each None or as its tensor (dx without an x:
    the gradient of h, which has h's type).  The other arguments are the forward
    call's; h and n are not needed.  dx may be dh itself, dy may be dn.  Returns
    the workspace."""
    args, M, D, index, x_type = _norm_args(y, None, None, x, gate, scale, post, post_weight, post_bias, pre, weight, bias, eps,
                                           stats)
    if stats is None:
        raise ValueError("the gradient needs the forward call's stats")
    if dh is None and dn is None:
        raise ValueError("neither dh nor dn is given")
    if dn is not None and pre is None:
        raise ValueError("dn without a pre-norm")
    if x is None and (dh is not None or dx is not None):
        x_type = (dh if dh is not None else dx).dtype
        if x_type not in (y.dtype, torch.float32):
            raise TypeError(f"dh has type {x_type}")
        args = (*args[:26], _DT[x_type], *args[27:])
    grads = [_like("dh", dh, (M, D), x_type, index), _like("dn", dn, (M, D), y.dtype, index),
             _like("dy", dy, (M, D), y.dtype, index), _like("dx", dx, (M, D), x_type, index)]
    if dgate is not None and gate is None:
        raise ValueError("dgate without a gate")
    grads.append(_NO_MAT if dgate is None else _like("dgate", dgate, tuple(gate.shape), gate.dtype, index))
    vectors = []
    for name, t, of in (("dpost_weight", dpost_weight, post_weight), ("dpost_bias", dpost_bias, post_bias),
                        ("dweight", dweight, weight), ("dbias", dbias, bias)):
        if t is not None and of is None:
            raise ValueError(f"{name} without its vector")
        vectors.append(0 if t is None else _vec(name, t, D, (of.dtype,), index))
    packed = _native.pack_norm_join_grad(*args, *(v for m in grads for v in m), *vectors)
    outs = [t for t in (dy, dx, dgate, dpost_weight, dpost_bias, dweight, dbias) if t is not None]
    return _sums("norm_join_grad", packed, outs, workspace, index, stream)


# ------------------------------------------------------------------ differentiable forms
# Their forward passes go through the ops above, with all of their checks; the
# backward passes' tensors are those, or made here, and are handed on as they are:
# autograd's threads run on cold caches, where each step costs three times as much.

def _rows(t: Optional[torch.Tensor], cols: int):
    """(..., cols) as a matrix; sizes of zero among them."""
    return t if t is None or t.dim() == 2 else t.reshape(math.prod(t.shape[:-1]), cols)


def _m(t: Optional[torch.Tensor]):
    """(data, row stride, column stride) of a matrix that needs no check."""
    return _NO_MAT if t is None else (t.data_ptr(), *t.stride())


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _graph_of(*tensors) -> bool:
    """Whether autograd has to see an op on these: it wants a node, or has tangents to refuse (these ops have no
    forward-mode derivatives)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    if forward_ad._current_level >= 0:  # within a dual level
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                return True
    return False


def _call(name: str, args, workspace, index: int) -> None:
    """A gradient's call with the caller's workspace, or the stream's."""
    ws = _layer_workspace(workspace, torch.device("cuda", index))
    _product(name, getattr(_native.load(), "iris_b200_" + name), args, None, None, ws, index, None)


def _linear(x, weight, bias, act, residual, p, rng, workspace, keep_z):
    """(y, z): the layer's output, and the activation's argument where it is to be kept."""
    K, N = weight.shape
    x2, dev = _rows(x, K), x.device
    y = torch.empty(x2.shape[0], N, dtype=x.dtype, device=dev)
    z = torch.empty(x2.shape[0], N, dtype=x.dtype, device=dev) if keep_z and act is not None else None
    matmul_act(x2, weight, y, bias=bias, act=act, residual=_rows(residual, N), z=z, p=p, rng=rng,
               workspace=_layer_workspace(workspace, dev))
    return (y if x.dim() == 2 else y.reshape(*x.shape[:-1], N)), z


class _LinearAct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, act, residual, p, rng, workspace):
        y, z = _linear(x, weight, bias, act, residual, p, rng, workspace, any(ctx.needs_input_grad[:3]))
        ctx.save_for_backward(x, weight, z, rng)
        ctx.args = _ACTS[act], p, workspace, None if bias is None else bias.dtype
        return y

    # the kernels' gradients have no derivatives of their own: asking for second
    # ones is an error, not a sum without some of its terms
    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, z, rng = ctx.saved_tensors
        act, p, workspace, bias_dtype = ctx.args
        want_x, want_w, want_b, _, want_r = ctx.needs_input_grad[:5]
        dx = dw = db = None
        if want_x or want_w or want_b:
            K, N = weight.shape
            x2, dy2, dev, dtype = _rows(x, K), _rows(dy, N), dy.device, x.dtype
            M = x2.shape[0]
            mdx = mdw = _NO_MAT
            if want_x:
                dx = torch.empty(x.shape, dtype=dtype, device=dev)
                mdx = dx.data_ptr(), K, 1
            if want_w:
                dw = torch.empty(K, N, dtype=dtype, device=dev)
                mdw = dw.data_ptr(), N, 1
            if want_b:
                db = torch.empty(N, dtype=bias_dtype, device=dev)
            args = _native.pack_linear_act_grad(*_m(dy2), *_m(x2), *_m(weight), *_m(z), *mdx, *mdw, _ptr(db), _ptr(rng), M, N, K, p,
                                                _DT[dtype], _DT[bias_dtype] if want_b else 0, act, 0)
            _call("linear_act_grad", args, workspace, dev.index)
        return dx, dw, db, None, dy if want_r else None, None, None, None


def linear_act(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, act: Optional[str] = None,
               residual: Optional[torch.Tensor] = None, p: float = 0.0, rng: Optional[torch.Tensor] = None, workspace=None):
    """Differentiable y = residual + dropout(act(x @ weight + bias)), x (..., K) and
    weight (K, N) f16 or bf16, residual (..., N) and y of the same type.

    Kept for the backward pass: x, weight, and with an activation its argument in
    16 bits; the gradient between the products is rounded to 16 bits, their
    operands' type, and lies in the workspace, which stays as large as that
    (2 bytes an element of the output) when the backward pass is done.  A
    workspace that is given serves forward and backward; else it is the stream's."""
    if x.dim() < 1 or x.dtype not in _DT16:
        raise TypeError("x is a f16 or bf16 tensor (..., K)")
    if not x.is_cuda:
        raise ValueError("x is not on a CUDA device")
    if weight.dim() != 2 or weight.dtype != x.dtype or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight is a {x.dtype} matrix of {x.shape[-1]} rows")
    if residual is not None and (residual.dtype != x.dtype or residual.shape != (*x.shape[:-1], weight.shape[1])):
        raise ValueError(f"residual is a {x.dtype} tensor of shape {(*x.shape[:-1], weight.shape[1])}")
    if not _graph_of(x, weight, bias, residual):
        return _linear(x, weight, bias, act, residual, p, rng, workspace, False)[0]
    return _LinearAct.apply(x, weight, bias, act, residual, p, rng, workspace)


def _dropped(x, p, rng, residual=None):
    N = x.shape[-1]
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dropout_add(_rows(x, N), _rows(out, N), p, rng, residual=_rows(residual, N))
    return out


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng, residual):
        ctx.save_for_backward(rng)
        ctx.p = p
        return _dropped(x, p, rng, residual)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        rng, = ctx.saved_tensors
        wants = ctx.needs_input_grad
        return _dropped(dy, ctx.p, rng) if wants[0] else None, None, None, dy if wants[3] else None


def dropout(x: torch.Tensor, p: float, rng: Optional[torch.Tensor], residual: Optional[torch.Tensor] = None):
    """Differentiable residual + dropout(x) of tensors (..., N).  Nothing is kept
    but rng, which must not change before the backward pass (autograd tells)."""
    if x.dim() < 1 or x.dtype not in _DT:
        raise TypeError("x is a f16, bf16 or f32 tensor (..., N)")
    if residual is not None and (residual.dtype != x.dtype or residual.shape != x.shape):
        raise ValueError(f"residual is a {x.dtype} tensor of shape {tuple(x.shape)}")
    if not _graph_of(x, residual):
        return _dropped(x, p, rng, residual)
    return _Dropout.apply(x, p, rng, residual)


def _joined(y, x, gate, post_weight, post_bias, weight, bias, scale, post, pre, eps, keep_stats):
    """(h, n, stats, the call's arguments); h None where nothing joins y, n without a pre-norm, stats where they are not to
    be kept."""
    D, dev = y.shape[-1], y.device
    y2, joins = _rows(y, D), x is not None or gate is not None or post is not None or scale != 1.0
    h = torch.empty(y.shape, dtype=(y if x is None else x).dtype, device=dev) if joins else None
    n = torch.empty(y.shape, dtype=y.dtype, device=dev) if pre is not None else None
    stats = torch.empty(y2.shape[0], 4, dtype=torch.float32, device=dev) if keep_stats else None
    args = _norm_join(y2, _rows(h, D), _rows(n, D), _rows(x, D), gate, scale, post, post_weight, post_bias, pre, weight, bias, eps,
                      stats)
    return h, n, stats, args


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, x, gate, post_weight, post_bias, weight, bias, scale, post, pre, eps, workspace):
        h, n, stats, args = _joined(y, x, gate, post_weight, post_bias, weight, bias, scale, post, pre, eps, True)
        ctx.save_for_backward(y, x, gate, post_weight, post_bias, weight, bias, stats)
        ctx.args = args, scale, post, pre, eps, workspace
        ctx.set_materialize_grads(False)
        return h, n

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dn):
        y, x, gate, post_weight, post_bias, weight, bias, stats = saved = ctx.saved_tensors
        args, scale, post, pre, eps, workspace = ctx.args
        if dh is None and dn is None:
            return (None,) * 12
        D, dev = y.shape[-1], y.device
        # what _rows copies has no other owner, so it is held here until the call has been made
        y2, x2, dh2, dn2 = _rows(y, D), _rows(x, D), _rows(dh, D), _rows(dn, D)
        grads = [torch.empty(t.shape, dtype=t.dtype, device=dev) if w and t is not None else None
                 for t, w in zip(saved[:7], ctx.needs_input_grad)]
        if pre is not None and dn is None:
            # n has had no part in the loss: its norm's vectors get no gradient
            grads[5] = grads[6] = None
            weight = bias = pre = None
        elif all(_m(t) == args[i:i + 3] for t, i in ((y2, 0), (x2, 3), (gate, 6))) and \
                all(_ptr(t) == args[i] for t, i in zip(saved[3:], range(15, 20))):
            # the tensors lie as the forward call found them (those that a hook on saved
            # ones has brought back may lie in the same place with other strides)
            mats = [_NO_MAT if t is None else (t.data_ptr(), D, 1) for t in grads[:3]]
            packed = _native.pack_norm_join_grad(*args, *_m(dh2), *_m(dn2), *mats[0], *mats[1], *mats[2],
                                                 *map(_ptr, grads[3:]))
            _call("norm_join_grad", packed, workspace, dev.index)
            return (*grads, None, None, None, None, None)
        dpost_weight, dpost_bias, dweight, dbias = grads[3:]
        norm_join_grad(y2, stats, dh2, dn2, x=x2, gate=gate, scale=scale, post=post,
                       post_weight=post_weight, post_bias=post_bias, pre=pre, weight=weight, bias=bias, eps=eps,
                       dy=_rows(grads[0], D), dx=_rows(grads[1], D), dgate=grads[2], dpost_weight=dpost_weight,
                       dpost_bias=dpost_bias, dweight=dweight, dbias=dbias, workspace=_layer_workspace(workspace, dev))
        return (*grads, None, None, None, None, None)


def block_norm(y: torch.Tensor, x: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
               post: Optional[str] = None, post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
               pre: Optional[str] = None, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-6, workspace=None):
    """Differentiable ``norm_join`` of tensors (..., D): returns (h, n), n None
    without a pre-norm, h y itself where nothing joins it.  gate (G, D) counts y's
    rows with the leading dimensions flattened; y, x and the gradients that come
    back are copied where their strides do not allow that.  Kept for the backward pass: the
    inputs and 4 numbers a row."""
    if y.dim() < 1 or y.dtype not in _DT:
        raise TypeError("y is a f16, bf16 or f32 tensor (..., D)")
    if x is not None and (x.dtype not in (y.dtype, torch.float32) or x.shape != y.shape):
        raise ValueError(f"x is a {y.dtype} or float32 tensor of shape {tuple(y.shape)}")
    if post is None and pre is None and x is None and gate is None and scale == 1.0:
        raise ValueError("nothing to do: no norm, residual, gate or scale")
    if _graph_of(y, x, gate, post_weight, post_bias, weight, bias):
        h, n = _BlockNorm.apply(y, x, gate, post_weight, post_bias, weight, bias, scale, post, pre, eps, workspace)
    else:
        h, n, _, _ = _joined(y, x, gate, post_weight, post_bias, weight, bias, scale, post, pre, eps, False)
    return (y if h is None else h), n
