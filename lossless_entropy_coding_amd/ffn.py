"""Feed-forward operators: matrix products with a fused epilogue (dense, or
grouped by expert) and layer norm, forward and backward.

Like the rest of the binding this module checks and marshals arguments; the
work runs in the library's HIP kernels, asynchronously on the current stream
(every function also takes ``stream=``).  Nothing is kept between calls: outputs and workspaces come
from torch's allocator, so the calls can be captured into a HIP graph.

Tensors are 2-D (or have their leading dimensions flattened by the caller),
rows may be strided, a row's elements are contiguous.  An e4m3 tensor is
``torch.float8_e4m3fn``; ``uint8`` is read as e4m3 bytes, so that what
``decode`` returns goes straight into a product.

Autograd does not see these calls: gradients come from the backward functions
here, called by the program.  A forward call warns where torch is recording
and a tensor requires its gradient, since the result will not.
"""

from __future__ import annotations

import ctypes
import functools
import warnings

import torch

_BF16, _E4M3, _FP32 = 1, 2, 3
_DTYPES = {torch.bfloat16: _BF16, torch.float8_e4m3fn: _E4M3, torch.uint8: _E4M3, torch.float32: _FP32}
_ACTS = {None: 0, "none": 0, "gelu": 1, "silu": 2, "relu": 3}
_FORWARD, _GRAD_INPUT, _GRAD_WEIGHT = 0, 1, 2

_vp, _u64, _u32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32


class _LinearArgs(ctypes.Structure):
    """ec_linear_args"""
    _fields_ = [
        ("m", _u64), ("n", _u64), ("k", _u64),
        ("groups", _u32), ("dtype", _u32), ("out_dtype", _u32), ("act", _u32),
        ("bias_dtype", _u32), ("x_scales", _u32), ("w_scales", _u32), ("reserved", _u32),
        ("offsets", _vp),
        ("x", _vp), ("x_stride", _u64),
        ("w", _vp), ("w_stride", _u64), ("w_group_stride", _u64),
        ("bias", _vp),
        ("residual", _vp), ("residual_stride", _u64),
        ("x_scale", _vp), ("w_scale", _vp), ("out_scale", _vp),
        ("y", _vp), ("y_stride", _u64),
        ("preact", _vp), ("preact_stride", _u64),
        ("dy", _vp), ("dy_stride", _u64),
        ("dx", _vp), ("dx_stride", _u64),
        ("dw", _vp), ("dw_stride", _u64), ("dw_group_stride", _u64),
        ("db", _vp),
        ("status", _vp),
        ("workspace", _vp), ("workspace_bytes", _u64),
    ]


_package = None


def _ec():
    global _package
    if _package is None:
        import lossless_entropy_coding_amd
        _package = lossless_entropy_coding_amd
    return _package


def _error(text: str):
    raise _ec().ECError(text)


def _matrix(t, name: str, rows: int, cols: int, dtypes, device=None):
    """Checks a 2-D CUDA tensor with contiguous rows; returns its row stride."""
    # one pass of cheap checks for what is in order: a call on one token takes as long as the host needs for it
    if isinstance(t, torch.Tensor) and t.is_cuda and t.shape == (rows, cols) and t.dtype in dtypes \
            and (device is None or t.device == device):
        s, one = t.stride()
        if one == 1 and s >= cols:
            return s
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        _error("%s must be a 2-D CUDA tensor" % name)
    if t.dtype not in dtypes:
        _error("%s must be %s, not %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.shape[0] != rows or t.shape[1] != cols:
        _error("%s must be [%d, %d], not %s" % (name, rows, cols, list(t.shape)))
    if device is not None and t.device != device:
        _error("%s is on %s, the other tensors on %s" % (name, t.device, device))
    return _row_stride(t, name)


def _row_stride(t, name: str) -> int:
    """Row stride (of the last two dimensions) in elements."""
    rows, cols = t.shape[-2], t.shape[-1]
    if cols > 1 and t.stride(-1) != 1:
        _error("%s must have contiguous rows" % name)
    s = t.stride(-2)
    if rows > 1 and s < cols:
        _error("%s has overlapping rows" % name)
    return max(s, cols)


def _vector(t, name: str, shapes, dtypes, device):
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and t.shape in shapes \
            and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.device != device or not t.is_contiguous():
        _error("%s must be a contiguous %s tensor on %s" % (name, " or ".join(str(d) for d in dtypes), device))
    if tuple(t.shape) not in shapes:
        _error("%s must have shape %s, not %s" % (name, " or ".join(str(list(s)) for s in shapes), list(t.shape)))


def _act(act) -> int:
    if act not in _ACTS:
        _error("act must be None, 'gelu', 'silu' or 'relu', not %r" % (act,))
    return _ACTS[act]


# straight from torch's C layer, a quarter of the time (public API as the fallback)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def _placed(fn):
    """``stream=s`` runs the call as under ``torch.cuda.stream(s)``: outputs
    and workspaces come from that stream's memory, so none is in use by work
    queued elsewhere.  The first tensor's device becomes the current one; a
    stream of another is refused."""

    first = fn.__code__.co_varnames[0]      # may be given by its name, like any other

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        t = args[0] if args else kw.get(first)
        if stream is not None:
            if isinstance(t, torch.Tensor) and t.is_cuda and stream.device != t.device:
                _error("stream is on %s, %s on %s" % (stream.device, first, t.device))
            with torch.cuda.stream(stream):
                return call(*args, **kw)
        if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != _current_device():
            with torch.cuda.device(t.device):
                return fn(*args, **kw)
        return fn(*args, **kw)

    return call


def _warn_unrecorded(level: int, *tensors):
    """`level`: frames between the caller's and this one."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                warnings.warn("autograd does not record this call: its result requires no gradient (use the backward "
                              "functions, and torch.no_grad() here)", stacklevel=level + 2)
                return


def _call(name: str, args: _LinearArgs, op: int, device):
    ec = _ec()
    L = ec.lib()
    need = int(L.linear_workspace_bytes(ctypes.byref(args), op))
    if need:  # freed at return, to be used again in the order of this stream
        ws = _empty(need, torch.uint8, device)
        args.workspace, args.workspace_bytes = ws.data_ptr(), need
    ec._check(getattr(L, name)(ctypes.byref(args), ec._stream(None)), name)


def _weights(w, name: str, offsets, dtypes):
    """(groups, n, k, row stride, group stride) of [n, k] or [groups, n, k] weights."""
    grouped = offsets is not None
    if not grouped and isinstance(w, torch.Tensor) and w.is_cuda and w.dim() == 2 and w.dtype in dtypes:
        (n, k), (s, one) = w.shape, w.stride()
        if one == 1 and s >= k:
            return 0, n, k, s, 0
    if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dim() != (3 if grouped else 2):
        _error("%s must be a %d-D CUDA tensor" % (name, 3 if grouped else 2))
    if w.dtype not in dtypes:
        _error("%s must be %s, not %s" % (name, " or ".join(str(d) for d in dtypes), w.dtype))
    groups = w.shape[0] if grouped else 0
    n, k = w.shape[-2:]
    stride = _row_stride(w, name)
    if grouped:
        if not 1 <= groups <= 4096:
            _error("%s must have 1 to 4096 groups" % name)
        if groups > 1 and n and k and w.stride(0) < (n - 1) * stride + k:
            _error("%s has overlapping groups" % name)
        if (not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or offsets.device != w.device
                or tuple(offsets.shape) != (groups + 1,) or not offsets.is_contiguous()):
            _error("offsets must be a contiguous int32 tensor of groups + 1 = %d entries on %s"
                   % (groups + 1, w.device))
    return groups, n, k, stride, (w.stride(0) if groups > 1 else 0)


def _given(t, name: str, dtype) -> None:
    """A tensor to write to that the caller has given, and the type asked for with it (or None)."""
    if not isinstance(t, torch.Tensor):
        _error("%s must be a tensor, not %s" % (name, type(t).__name__))
    if dtype is not None and t.dtype != dtype:
        _error("%s is %s, %s_dtype %s" % (name, t.dtype, name, dtype))


def _status(status, device):
    if status is None:
        return None
    if not isinstance(status, torch.Tensor) or status.dtype != torch.int32 or status.device != device or status.numel() < 1:
        _error("status must be an int32 tensor on %s" % device)
    return status.data_ptr()


def _forward(x, w, offsets, bias, act, residual, x_scale, w_scale, out_scale, out_dtype, save_preact, out, preact,
             status):
    E4 = (torch.float8_e4m3fn, torch.uint8)
    a = _LinearArgs()
    a.groups, n, k, a.w_stride, a.w_group_stride = _weights(w, "w", offsets, (torch.bfloat16,) + E4)
    dev = w.device
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _error("x must be a 2-D CUDA tensor")
    m = x.shape[0]
    a.x_stride = _matrix(x, "x", m, k, (torch.bfloat16,) if w.dtype == torch.bfloat16 else E4, dev)
    a.m, a.n, a.k = m, n, k
    a.dtype = _DTYPES[w.dtype]
    a.act = _act(act)
    a.x, a.w = x.data_ptr(), w.data_ptr()
    per = (a.groups,) if a.groups else ()
    if a.groups:
        a.offsets = offsets.data_ptr()
        a.status = _status(status, dev)
    if bias is not None:
        _vector(bias, "bias", (per + (n,),), (torch.float32, torch.bfloat16), dev)
        a.bias, a.bias_dtype = bias.data_ptr(), _DTYPES[bias.dtype]
    if residual is not None:
        a.residual_stride = _matrix(residual, "residual", m, n, (torch.bfloat16,), dev)
        a.residual = residual.data_ptr()
    if x_scale is not None:
        _vector(x_scale, "x_scale", ((1,), (m,)), (torch.float32,), dev)
        a.x_scale, a.x_scales = x_scale.data_ptr(), x_scale.numel()
    if w_scale is not None:
        _vector(w_scale, "w_scale", (per + (1,), per + (n,)), (torch.float32,), dev)
        a.w_scale, a.w_scales = w_scale.data_ptr(), w_scale.shape[-1]
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16
        if out_dtype not in _DTYPES:
            _error("out_dtype must be bfloat16, float32, float8_e4m3fn or uint8 (e4m3 bytes), not %s" % out_dtype)
        out, a.y_stride = _empty((m, n), out_dtype, dev), n
    else:
        _given(out, "out", out_dtype)
        a.y_stride = _matrix(out, "out", m, n, _DTYPES, dev)
    a.y, a.out_dtype = out.data_ptr(), _DTYPES[out.dtype]
    if out_scale is not None:
        if a.out_dtype != _E4M3:
            _error("out_scale goes with an e4m3 output")
        _vector(out_scale, "out_scale", ((1,),), (torch.float32,), dev)
        a.out_scale = out_scale.data_ptr()
    if save_preact or preact is not None:
        if preact is None:
            preact, a.preact_stride = _empty((m, n), torch.bfloat16, dev), n
        else:
            a.preact_stride = _matrix(preact, "preact", m, n, (torch.bfloat16,), dev)
        a.preact = preact.data_ptr()
    _warn_unrecorded(3, x, w, bias, residual)
    _call("linear_forward", a, _FORWARD, dev)
    return out if preact is None else (out, preact)


@_placed
def linear(x, w, bias=None, *, act=None, residual=None, x_scale=None, w_scale=None, out_scale=None, out_dtype=None,
           save_preact=False, out=None, preact=None):
    """y = act(x w^T * x_scale * w_scale + bias) + residual.

    x [m, k] and w [n, k] both bfloat16, or both e4m3.  bias [n] float32 or
    bfloat16; act None, 'gelu' (erf form), 'silu' or 'relu'; residual [m, n]
    bfloat16.  x_scale float32 [1] or [m] (one per row), w_scale [1] or [n].
    out_dtype bfloat16 (default), float32, float8_e4m3fn or uint8 (e4m3
    bytes, ready for ``encode``); an e4m3 result is multiplied by out_scale
    (float32 [1]) first and saturates at 448.

    Returns y, or (y, preact) with save_preact (or a preact buffer): the
    activation's input as bfloat16, for the backward pass."""
    return _forward(x, w, None, bias, act, residual, x_scale, w_scale, out_scale, out_dtype, save_preact, out, preact,
                    None)


@_placed
def grouped_linear(x, w, offsets, bias=None, *, act=None, residual=None, x_scale=None, w_scale=None, out_scale=None,
                   out_dtype=None, save_preact=False, out=None, preact=None, status=None):
    """``linear`` by expert: rows offsets[e] .. offsets[e + 1] - 1 of x go
    through w[e] ([groups, n, k]), bias[e] and w_scale[e].

    offsets is an int32 CUDA tensor of groups + 1 entries that never
    decrease, read on the GPU only; groups may be empty, and rows of no group
    get zeros.  Offsets out of order or range set S_BAD_OFFSETS in status
    (int32 [1], optional)."""
    if offsets is None:
        _error("offsets must be a tensor")
    return _forward(x, w, offsets, bias, act, residual, x_scale, w_scale, out_scale, out_dtype, save_preact, out,
                    preact, status)


def _backward(dy, x, w, offsets, preact, act, need_dx, need_dw, need_db, dw_dtype, dx, dw, db, status):
    bf = (torch.bfloat16,)
    groups, n, k, w_stride, w_group = _weights(w, "w", offsets, bf)
    dev = w.device
    if not isinstance(dy, torch.Tensor) or dy.dim() != 2:
        _error("dy must be a 2-D CUDA tensor")
    m = dy.shape[0]
    a = _LinearArgs()
    a.m, a.n, a.k, a.groups, a.dtype = m, n, k, groups, _BF16
    a.dy_stride, a.dy = _matrix(dy, "dy", m, n, bf, dev), dy.data_ptr()
    if groups:
        a.offsets = offsets.data_ptr()
        a.status = _status(status, dev)
    per = (groups,) if groups else ()
    need_dx, need_dw, need_db = need_dx or dx is not None, need_dw or dw is not None, need_db or db is not None
    a.act = _act(act)
    if need_dx:
        a.w, a.w_stride, a.w_group_stride = w.data_ptr(), w_stride, w_group
        if a.act:
            if preact is None:
                _error("preact (the activation's input) is needed for the gradient through act")
            a.preact_stride, a.preact = _matrix(preact, "preact", m, k, bf, dev), preact.data_ptr()
        if dx is None:
            dx, a.dx_stride = _empty((m, k), torch.bfloat16, dev), k
        else:
            a.dx_stride = _matrix(dx, "dx", m, k, bf, dev)
        a.dx = dx.data_ptr()
        _call("linear_grad_input", a, _GRAD_INPUT, dev)
    if need_dw or need_db:
        if need_dw:
            a.x_stride, a.x = _matrix(x, "x", m, k, bf, dev), x.data_ptr()
            if dw is None:
                dw = _empty(per + (n, k), dw_dtype if dw_dtype is not None else torch.bfloat16, dev)
            else:
                _given(dw, "dw", dw_dtype)
            if tuple(dw.shape) != per + (n, k) or dw.device != dev:
                _error("dw must be %s on %s" % (list(per + (n, k)), dev))
            if dw.dtype not in (torch.bfloat16, torch.float32):
                _error("dw must be bfloat16 or float32, not %s" % dw.dtype)
            a.dw_stride, a.dw, a.out_dtype = _row_stride(dw, "dw"), dw.data_ptr(), _DTYPES[dw.dtype]
            a.dw_group_stride = dw.stride(0) if groups > 1 else 0
        if need_db:
            if db is None:
                db = _empty(per + (n,), torch.float32, dev)
            else:
                _vector(db, "db", (per + (n,),), (torch.float32,), dev)
            a.db = db.data_ptr()
        _call("linear_grad_weight", a, _GRAD_WEIGHT, dev)
    return dx, dw, db


@_placed
def linear_backward(dy, x, w, *, preact=None, act=None, need_dx=True, need_dw=True, need_db=True, dw_dtype=None,
                    dx=None, dw=None, db=None):
    """Gradients of ``x w^T + bias`` for dy [m, n] (bfloat16).

    Returns (dx, dw, db), None where not needed:
      dx [m, k] bfloat16 = (dy w) * act'(preact), where x = act(preact): the
         gradient goes straight through the activation that made x (act None:
         dx = dy w);
      dw [n, k] = dy^T x in dw_dtype (bfloat16, or float32);
      db [n] float32 = sum of dy's rows.
    Sums run in a fixed order: the same call gives the same bits."""
    return _backward(dy, x, w, None, preact, act, need_dx, need_dw, need_db, dw_dtype, dx, dw, db, None)


@_placed
def grouped_linear_backward(dy, x, w, offsets, *, preact=None, act=None, need_dx=True, need_dw=True, need_db=True,
                            dw_dtype=None, dx=None, dw=None, db=None, status=None):
    """``linear_backward`` by expert: dw [groups, n, k] and db [groups, n]
    hold each expert's sums over its rows (zeros for an empty one); rows of
    no group get zeros in dx."""
    if offsets is None:
        _error("offsets must be a tensor")
    return _backward(dy, x, w, offsets, preact, act, need_dx, need_dw, need_db, dw_dtype, dx, dw, db, status)


def _norm_params(weight, bias, cols, dev):
    kinds = (torch.float32, torch.bfloat16)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _vector(t, name, ((cols,),), kinds, dev)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        _error("weight and bias must have one type")
    given = weight if weight is not None else bias
    return _DTYPES[given.dtype] if given is not None else _FP32


def _ptr(t):
    return None if t is None else t.data_ptr()


@_placed
def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, out_dtype=None, out_scale=None, out=None, mean=None,
               rstd=None):
    """Layer norm over the last dimension of x [rows, cols] (bfloat16 or
    float32): y = (x - mean) * rstd * weight + bias.

    weight, bias [cols] float32 or bfloat16.  out_dtype: x's (default),
    bfloat16, float32, float8_e4m3fn or uint8 (e4m3 bytes; multiplied by
    out_scale first, saturating).  Returns (y, mean, rstd), the last two
    float32 [rows] for the backward pass."""
    ec = _ec()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _error("x must be a 2-D CUDA tensor")
    rows, cols = x.shape
    xs = _matrix(x, "x", rows, cols, (torch.bfloat16, torch.float32))
    dev = x.device
    if not 1 <= cols <= 65536:
        _error("x must have 1 to 65536 columns")
    w_dtype = _norm_params(weight, bias, cols, dev)
    if out is None:
        out_dtype = x.dtype if out_dtype is None else out_dtype
        if out_dtype not in _DTYPES:
            _error("out_dtype must be bfloat16, float32, float8_e4m3fn or uint8 (e4m3 bytes), not %s" % out_dtype)
        out, ys = _empty((rows, cols), out_dtype, dev), cols
    else:
        _given(out, "out", out_dtype)
        ys = _matrix(out, "out", rows, cols, _DTYPES, dev)
    if out_scale is not None:
        if _DTYPES[out.dtype] != _E4M3:
            _error("out_scale goes with an e4m3 output")
        _vector(out_scale, "out_scale", ((1,),), (torch.float32,), dev)
    if mean is None and rstd is None:
        mean, rstd = _empty((rows,), torch.float32, dev), _empty((rows,), torch.float32, dev)
    else:
        for t, name in ((mean, "mean"), (rstd, "rstd")):
            _vector(t, name, ((rows,),), (torch.float32,), dev)
    _warn_unrecorded(2, x, weight, bias)
    ec._check(ec.lib().layer_norm_forward(x.data_ptr(), _DTYPES[x.dtype], rows, cols, xs, _ptr(weight), _ptr(bias),
                                          w_dtype, float(eps), out.data_ptr(), _DTYPES[out.dtype], ys,
                                          _ptr(out_scale), mean.data_ptr(), rstd.data_ptr(), ec._stream(None)),
              "layer_norm_forward")
    return out, mean, rstd


@_placed
def layer_norm_backward(dy, x, mean, rstd, weight=None, *, residual_grad=None, need_dx=True, need_dweight=True,
                        need_dbias=True, dx=None, dweight=None, dbias=None):
    """Backward of ``layer_norm`` for dy [rows, cols] of x's type.

    Returns (dx, dweight, dbias), None where not needed.  residual_grad (x's
    type) is added to dx: the gradient that reaches x past the norm.  dweight
    and dbias are float32 [cols], summed in a fixed order.  dx may be dy, x or
    residual_grad itself, beyond 8192 columns only the last."""
    ec = _ec()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _error("x must be a 2-D CUDA tensor")
    rows, cols = x.shape
    xs = _matrix(x, "x", rows, cols, (torch.bfloat16, torch.float32))
    dev = x.device
    if not 1 <= cols <= 65536:
        _error("x must have 1 to 65536 columns")
    same = (x.dtype,)
    ds = _matrix(dy, "dy", rows, cols, same, dev)
    w_dtype = _norm_params(weight, None, cols, dev)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _vector(t, name, ((rows,),), (torch.float32,), dev)
    rs = _matrix(residual_grad, "residual_grad", rows, cols, same, dev) if residual_grad is not None else 0
    need_dx, need_dweight, need_dbias = need_dx or dx is not None, need_dweight or dweight is not None, \
        need_dbias or dbias is not None
    xds = 0
    if need_dx:
        if dx is None:
            dx, xds = _empty((rows, cols), x.dtype, dev), cols
        else:
            xds = _matrix(dx, "dx", rows, cols, same, dev)
    if need_dweight:
        if dweight is None:
            dweight = _empty((cols,), torch.float32, dev)
        else:
            _vector(dweight, "dweight", ((cols,),), (torch.float32,), dev)
    if need_dbias:
        if dbias is None:
            dbias = _empty((cols,), torch.float32, dev)
        else:
            _vector(dbias, "dbias", ((cols,),), (torch.float32,), dev)
    L = ec.lib()
    ws, need = None, 0
    if need_dweight or need_dbias:
        need = int(L.layer_norm_grad_workspace_bytes(rows, cols))
        ws = _empty(need, torch.uint8, dev)
    ec._check(L.layer_norm_grad(dy.data_ptr(), ds, x.data_ptr(), xs, _DTYPES[x.dtype], rows, cols, mean.data_ptr(),
                                rstd.data_ptr(), _ptr(weight), w_dtype, _ptr(residual_grad), rs, _ptr(dx), xds,
                                _ptr(dweight), _ptr(dbias), _ptr(ws), need, ec._stream(None)), "layer_norm_grad")
    return dx, dweight, dbias
