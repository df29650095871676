"""What a training step needs around its layers: the loss over a vocabulary,
with its gradients, and the weight update over many tensors.

Like ``ffn`` this module checks and marshals arguments; the work runs in the
library's HIP kernels, asynchronously on the current stream (``stream=`` for
another).  Nothing is kept between calls, and all that changes from step to
step (the step's number, gradients, a learning rate given as a tensor) is read
on the GPU, so that the calls can be captured into a HIP graph and replayed.
"""

from __future__ import annotations

import array
import ctypes
import math
import struct
from typing import NamedTuple, Optional

import torch

from .ffn import (_BF16, _DTYPES, _E4M3, _FP32, _current_device, _ec, _empty, _error, _given, _matrix, _placed, _row_stride,
                  _run, _status, _vector, _warn_unrecorded)

_vp, _u64, _u32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32


class _LossArgs(ctypes.Structure):
    """ec_loss_args"""
    _fields_ = [
        ("m", _u64), ("n", _u64), ("k", _u64),
        ("x", _vp), ("x_stride", _u64),
        ("w", _vp), ("w_stride", _u64),
        ("target", _vp), ("target_bytes", _u32), ("dlosses", _u32), ("ignore_index", ctypes.c_int64),
        ("loss", _vp), ("lse", _vp), ("dloss", _vp),
        ("dx", _vp), ("dx_stride", _u64),
        ("dw", _vp), ("dw_stride", _u64), ("dw_dtype", _u32), ("reserved", _u32),
        ("status", _vp),
        ("workspace", _vp), ("workspace_bytes", _u64),
    ]


def _loss_args(x, w, target, ignore_index, status):
    bf = (torch.bfloat16,)
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _error("x must be a 2-D CUDA tensor")
    m, k = x.shape
    a = _LossArgs()
    a.x_stride, a.x = _matrix(x, "x", m, k, bf), x.data_ptr()
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        _error("w must be a 2-D CUDA tensor")
    n, dev = w.shape[0], x.device
    if n < 1:
        _error("w must have a row")
    a.w_stride, a.w = _matrix(w, "w", n, k, bf, dev), w.data_ptr()
    _vector(target, "target", ((m,),), (torch.int64, torch.int32), dev)
    a.target, a.target_bytes = target.data_ptr(), target.element_size()
    if not isinstance(ignore_index, int) or not -(1 << 63) <= ignore_index < 1 << 63:
        _error("ignore_index must be a whole number of 64 bits, not %r" % (ignore_index,))
    a.ignore_index = ignore_index
    a.m, a.n, a.k = m, n, k
    a.status = _status(status, dev)
    return a, m, n, k, dev


@_placed
def linear_cross_entropy(x, w, target, *, ignore_index=-100, loss=None, lse=None, status=None):
    """Softmax cross entropy of the logits x w^T, which are never kept.

    x [m, k] and w [n, k] bfloat16 (n entries of the vocabulary), target [m]
    int64 or int32.  Returns (loss, lse), both float32 [m]: loss = lse - the
    target's logit, with lse = log of the sum of the row's exponentials, which
    the backward pass needs.  Rows whose target is ignore_index have loss 0;
    so have those with a target outside [0, n), which set S_BAD_TARGET in
    status (int32 [1], optional)."""
    a, m, n, k, dev = _loss_args(x, w, target, ignore_index, status)
    if loss is None:
        loss = _empty((m,), torch.float32, dev)
    else:
        _vector(loss, "loss", ((m,),), (torch.float32,), dev)
    if lse is None:
        lse = _empty((m,), torch.float32, dev)
    else:
        _vector(lse, "lse", ((m,),), (torch.float32,), dev)
    a.loss, a.lse = loss.data_ptr(), lse.data_ptr()
    _warn_unrecorded(2, x, w)
    _run("linear_cross_entropy_workspace_bytes", "linear_cross_entropy", a, dev)
    return loss, lse


@_placed
def linear_cross_entropy_backward(dloss, x, w, target, lse, *, ignore_index=-100, need_dx=True, need_dw=True,
                                  dw_dtype=None, dx=None, dw=None, status=None):
    """Gradients of ``linear_cross_entropy`` for dloss (float32 [m], or [1]
    for every row), from its lse.

    Returns (dx, dw), None where not needed: dx [m, k] bfloat16, dw [n, k] in
    dw_dtype (bfloat16, or float32).  Rows without a target get zeros in dx
    and add nothing to dw, whatever x holds there.  The logits are computed
    again by pieces of the vocabulary, and their gradient is rounded to
    bfloat16 for the two products.  Sums run in a fixed order: the same call
    gives the same bits.  Buffers given for the results overlap nothing that is
    read."""
    if not isinstance(dloss, torch.Tensor) or not dloss.is_cuda:
        _error("dloss must be a CUDA tensor")
    a, m, n, k, dev = _loss_args(x, w, target, ignore_index, status)
    _vector(dloss, "dloss", ((1,), (m,)), (torch.float32,), dev)
    a.dloss, a.dlosses = dloss.data_ptr(), dloss.numel()
    _vector(lse, "lse", ((m,),), (torch.float32,), dev)
    a.lse = lse.data_ptr()
    if need_dx or dx is not None:
        if dx is None:
            dx, a.dx_stride = _empty((m, k), torch.bfloat16, dev), k
        else:
            a.dx_stride = _matrix(dx, "dx", m, k, (torch.bfloat16,), dev)
        a.dx = dx.data_ptr()
    if need_dw or dw is not None:
        if dw is None:
            dw = _empty((n, k), dw_dtype if dw_dtype is not None else torch.bfloat16, dev)
        else:
            _given(dw, "dw", dw_dtype)
        if tuple(dw.shape) != (n, k) or dw.device != dev:
            _error("dw must be %s on %s" % ([n, k], dev))
        if dw.dtype not in (torch.bfloat16, torch.float32):
            _error("dw must be bfloat16 or float32, not %s" % dw.dtype)
        a.dw_stride, a.dw, a.dw_dtype = _row_stride(dw, "dw"), dw.data_ptr(), _DTYPES[dw.dtype]
    if dx is not None or dw is not None:
        _run("linear_cross_entropy_grad_workspace_bytes", "linear_cross_entropy_grad", a, dev)
    return dx, dw


# ------------------------------------------------------------------------ AdamW

ADAMW_BLOCK = 256


class _AdamWTensor(ctypes.Structure):
    """ec_adamw_tensor"""
    _fields_ = [("param", _vp), ("grad", _vp), ("copy", _vp), ("n", _u64), ("grad_dtype", _u32),
                ("weight_decay", ctypes.c_float)]


class _AdamWArgs(ctypes.Structure):
    """ec_adamw_args"""
    _fields_ = [
        ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp), ("state_blocks", _u64), ("steps", _vp), ("lr_at", _vp),
        ("grad_scale", _vp), ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double), ("state_dtype", _u32), ("seed", _u32),
    ]


class AdamWState(NamedTuple):
    """What ``adamw`` keeps of a list of tensors, one after the other in blocks
    of 256 values (a tensor begins a block; what its last block holds past its
    end is zero).

    m, v: both float32, or both e4m3 (``torch.float8_e4m3fn``; ``uint8`` is
    read as e4m3 bytes), [256 blocks].  In e4m3, m is the mean of the
    gradients over m_scale of its block, v the root of the mean of their
    squares over v_scale; m_scale, v_scale float32 [blocks], powers of two
    (None for float32 states).  steps int32 [1]: steps done."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: Optional[torch.Tensor]
    v_scale: Optional[torch.Tensor]
    steps: torch.Tensor


def _blocks(n: int) -> int:
    return -(-n // ADAMW_BLOCK)


def _params(params):
    if not isinstance(params, (list, tuple)) or not params:
        _error("params must be a list or tuple of tensors")
    for p in params:
        if not isinstance(p, torch.Tensor) or not p.is_cuda or p.dtype != torch.float32 or not p.is_contiguous():
            _error("params must be contiguous float32 CUDA tensors")


def adamw_state(params, state_dtype=torch.float32) -> AdamWState:
    """The state of ``adamw`` before the first step: zeros, float32 or
    (state_dtype float8_e4m3fn or uint8) e4m3."""
    _params(params)
    if state_dtype not in (torch.float32, torch.float8_e4m3fn, torch.uint8):
        _error("state_dtype must be float32, float8_e4m3fn or uint8 (e4m3 bytes), not %s" % state_dtype)
    blocks, dev = sum(_blocks(p.numel()) for p in params), params[0].device
    if any(p.device != dev for p in params):
        _error("params must be on one device")
    n, coded = blocks * ADAMW_BLOCK, state_dtype != torch.float32

    def zeros():
        if not coded:
            return torch.zeros(n, dtype=torch.float32, device=dev)
        return torch.zeros(n, dtype=torch.uint8, device=dev).view(state_dtype)

    def ones():
        return torch.full((blocks,), 2.0 ** -60, device=dev) if coded else None

    return AdamWState(zeros(), zeros(), ones(), ones(), torch.zeros(1, dtype=torch.int32, device=dev))


def _number(v, name: str, least, below=math.inf) -> float:
    v = float(v)
    if not least <= v < below:
        _error("%s must be %s, not %r" % (name, "at least %g" % least if below == math.inf else "in [%g, %g)" % (least, below), v))
    return v


_STATES = (torch.float32, torch.float8_e4m3fn, torch.uint8)


def _float_bits(v: float) -> int:
    return struct.unpack("<I", struct.pack("<f", v))[0]


def _once(places, sizes, name: str):
    """Refuses a tensor that is listed twice (tied weights): two writers of one place."""
    held = [p for p, n in zip(places, sizes) if p and n]
    if len(set(held)) != len(held):
        _error("%s must not hold the same tensor twice (tied weights are listed once, with the sum of their gradients)" % name)


def _bad_param(p, dev):
    _params([p])
    _error("params are on %s and %s" % (dev, p.device))


def adamw(params, grads, state: AdamWState, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=None,
          copies=None, seed=0, stream=None):
    """One step of AdamW (decoupled weight decay) over all params at once, in
    place.

    params: contiguous float32 tensors of any shapes on one device; grads: one
    for each, contiguous, of as many values, bfloat16 or float32 (as the
    backward functions give them); state: ``adamw_state(params)``, updated in place, its step
    number too.  lr a number, or a float32 [1] tensor read on the GPU;
    weight_decay a number or one for each tensor; grad_scale float32 [1]
    multiplies the gradients (what clipping their norm gives).  copies:
    bfloat16 tensors, or None for some, that get the new params rounded, the
    weights that the layers work with.

    States in e4m3 are rounded up or down at random, so that their means are
    kept: by a function of seed (32 bits), the step's number and the place, so
    that the same call gives the same bits.  Values that are not finite become
    NaN there.  Where v is held as 0 beside much larger values of its block, the
    step takes the least root that can be held (2^-9 v_scale), so that such a
    value moves by a few lr at most.  No two tensors may overlap."""
    if not isinstance(params, (list, tuple)) or not params or not isinstance(params[0], torch.Tensor) or not params[0].is_cuda:
        _params(params)
    if stream is not None and stream.device != params[0].device:
        _error("stream is on %s, params on %s" % (stream.device, params[0].device))
    index = params[0].get_device()
    if stream is not None or index != _current_device():
        with torch.cuda.stream(stream), torch.cuda.device(index):
            return adamw(params, grads, state, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, grad_scale=grad_scale,
                         copies=copies, seed=seed)
    count, dev = len(params), params[0].device
    if not isinstance(grads, (list, tuple)) or len(grads) != count:
        _error("grads must be a list or tuple of %d, one for each of params" % count)
    if copies is not None and (not isinstance(copies, (list, tuple)) or len(copies) != count):
        _error("copies must be a list or tuple of %d, one for each of params" % count)
    if isinstance(weight_decay, (list, tuple)):
        if len(weight_decay) != count:
            _error("weight_decay must be a number or one for each of params (%d)" % count)
        decays = [_float_bits(_number(d, "weight_decay", 0.0, 1e38)) << 32 for d in weight_decay]
    else:
        decays = [_float_bits(_number(weight_decay, "weight_decay", 0.0, 1e38)) << 32] * count
    # one pass of cheap checks: a step of small tensors takes as long as the host needs for it
    words, blocks = [], 0                       # ec_adamw_tensor's, five of 64 bits
    fp32, bf16, Tensor = torch.float32, torch.bfloat16, torch.Tensor
    for p, g, c, decay in zip(params, grads, copies if copies is not None else [None] * count, decays):
        if not (isinstance(p, Tensor) and p.dtype is fp32 and p.get_device() == index and p.is_contiguous()):
            _bad_param(p, dev)
        n = p.numel()
        if not (isinstance(g, Tensor) and g.get_device() == index and g.numel() == n and g.is_contiguous()):
            _error("grads must be contiguous tensors on %s of as many values as params" % dev)
        kind = g.dtype
        if kind is bf16:
            decay |= _BF16
        elif kind is fp32:
            decay |= _FP32
        else:
            _error("grads must be bfloat16 or float32, not %s" % kind)
        copy = 0
        if c is not None:
            if not (isinstance(c, Tensor) and c.dtype is bf16 and c.get_device() == index and c.numel() == n
                    and c.is_contiguous()):
                _error("copies must be contiguous bfloat16 tensors on %s of as many values as params, or None" % dev)
            copy = c.data_ptr()
        words += (p.data_ptr(), g.data_ptr(), copy, n, decay)
        blocks += (n + 255) >> 8
    if len(set(words[::5])) != count or copies is not None:
        _once(words[::5], words[3::5], "params")
        _once(words[2::5], words[3::5], "copies")
    if not isinstance(state, (list, tuple)) or len(state) != 5:
        _error("state must be an AdamWState")
    m, v, m_scale, v_scale, steps = state
    length = ((blocks * ADAMW_BLOCK,),)
    _vector(m, "state.m", length, _STATES, dev)
    _vector(v, "state.v", length, _STATES, dev)
    kind = _DTYPES[m.dtype]
    if _DTYPES[v.dtype] != kind:
        _error("state.m is %s, state.v %s" % (m.dtype, v.dtype))
    scales = (None, None)
    if kind == _E4M3:
        _vector(m_scale, "state.m_scale", ((blocks,),), (fp32,), dev)
        _vector(v_scale, "state.v_scale", ((blocks,),), (fp32,), dev)
        scales = m_scale.data_ptr(), v_scale.data_ptr()
    _vector(steps, "state.steps", ((1,),), (torch.int32,), dev)
    lr_at = None
    if isinstance(lr, Tensor):
        _vector(lr, "lr", ((1,),), (fp32,), dev)
        lr, lr_at = 0.0, lr.data_ptr()
    if grad_scale is not None:
        _vector(grad_scale, "grad_scale", ((1,),), (fp32,), dev)
        grad_scale = grad_scale.data_ptr()
    if not isinstance(seed, int) or not 0 <= seed < 1 << 32:
        _error("seed must be a whole number of 32 bits, not %r" % (seed,))
    if not isinstance(betas, (list, tuple)) or len(betas) != 2:
        _error("betas must be two numbers")
    beta1, beta2 = betas
    a = _AdamWArgs(m.data_ptr(), v.data_ptr(), *scales, blocks, steps.data_ptr(), lr_at, grad_scale, _number(lr, "lr", 0.0, 1e38),
                   _number(beta1, "betas[0]", 0.0, 1.0), _number(beta2, "betas[1]", 0.0, 1.0), _number(eps, "eps", 0.0, 1e38), kind,
                   seed)
    ec = _ec()
    tensors = array.array("Q", words)
    ec._check(ec.lib().adamw_step(tensors.buffer_info()[0], count, ctypes.byref(a), ec._stream(None)), "adamw_step")
