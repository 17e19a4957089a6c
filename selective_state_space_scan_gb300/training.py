"""Python binding of the calls that train a stack of layers next to the scan's own: layer norm and
convolution with their backward passes, and the losses over the vocabulary with their gradients.

Argument marshalling only, as in the package's other calls; ``include/selscan.h`` has the
definitions.  Workspaces are scratch of a single call, from PyTorch's allocator on the call's stream:
calls on several streams, from several threads or in several graphs share none.
"""
from __future__ import annotations

import ctypes

import selective_state_space_scan_gb300 as _ss

from .serving import _cuda, _empty, _io, _load, _norm_args, _param, _rows, _stream

_WS_BYTES = {}


def _scratch(t, stream, call, *sizes):
    """Workspace of one call (its memory may be handed on as soon as the call's work is on the stream).  Its bytes are
    asked for once for every device and sizes (the plan depends on the device's SM count)."""
    key = (call, t.get_device(), sizes)
    n = _WS_BYTES.get(key)
    if n is None:
        n = _ss._remember(_WS_BYTES, key, max(1, int(getattr(_ss.lib(), call)(*sizes))))
    return _empty((n,), _load().uint8, t.device, stream), n


def ss_add_layernorm(x, weight, bias=None, residual=None, eps=1e-5, y=None, residual_out=None, stream=None):
    """r = x + residual, y = (r - mean(r)) / sqrt(var(r) + eps) * weight + bias over rows (ss_add_layernorm).

    x [rows, D] and residual [rows, D]: float32 or bfloat16, each its own; weight, bias [D] float32.
    Returns (y, residual_out, mean, rstd): y like x, r in the residual's type (residual_out may be
    residual; without a residual it is x itself), and the rows' statistics [rows] float32 for
    ss_add_layernorm_bwd."""
    torch = _load()
    if residual is None and residual_out is None:
        _cuda(x, "x")
        rows, D = shape = x.shape
        dtype = x.dtype
        if y is None:
            y = _empty(shape, dtype, x.device, stream)
        s = _ss.NormStrides(_io(dtype), _io(dtype), _rows(x, "x", dtype, shape), 0, 0, _rows(y, "y", dtype, shape))
        _param(weight, "weight", torch.float32, (D,))
        r, out = x, None
    else:
        rows, D, out, y, s = _norm_args(x, weight, residual, residual_out, y, None, stream)
        r = out
    _param(bias, "bias", torch.float32, (D,))
    mean, rstd = _empty((rows,), torch.float32, x.device, stream), _empty((rows,), torch.float32, x.device, stream)
    st = _ss.lib().ss_add_layernorm(x.data_ptr(), _ss._ptr(residual), weight.data_ptr(), _ss._ptr(bias), _ss._ptr(out), y.data_ptr(),
                                    mean.data_ptr(), rstd.data_ptr(), rows, D, eps, ctypes.byref(s), _stream(x, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_add_layernorm")
    return y, r, mean, rstd


def ss_add_layernorm_bwd(dy, r, weight, mean, rstd, dr=None, stream=None):
    """Gradients of ss_add_layernorm (ss_add_layernorm_bwd): dy [rows, D] the gradient of y, r, mean and
    rstd from the forward call, dr [rows, D] the gradient of r from the layers behind (r's type) or None.

    Returns a dict: dx like dy, dresidual like r (the same tensor where the types are equal: both are the
    gradient of x + residual), dweight and dbias [D] float32."""
    torch = _load()
    _cuda(dy, "dy")
    rows, D = shape = dy.shape
    io, rdt, f32 = dy.dtype, r.dtype, torch.float32
    s = _ss.NormGradStrides(_io(io), _io(rdt), _rows(dy, "dy", io, shape), _rows(dr, "dr", rdt, shape), _rows(r, "r", rdt, shape), D, D)
    _param(weight, "weight", f32, (D,))
    _param(mean, "mean", f32, (rows,))
    _param(rstd, "rstd", f32, (rows,))
    dev = dy.device
    dx = _empty(shape, io, dev, stream)
    dres = dx if rdt is io else _empty(shape, rdt, dev, stream)
    dweight, dbias = _empty((D,), f32, dev, stream), _empty((D,), f32, dev, stream)
    ws, nbytes = _scratch(dy, stream, "ss_add_layernorm_bwd_workspace_size", rows, D)
    st = _ss.lib().ss_add_layernorm_bwd(dy.data_ptr(), _ss._ptr(dr), r.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                        dx.data_ptr(), None if dres is dx else dres.data_ptr(), dweight.data_ptr(), dbias.data_ptr(),
                                        rows, D, ctypes.byref(s), ws.data_ptr(), nbytes, _stream(dy, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_add_layernorm_bwd")
    return dict(dx=dx, dresidual=dres, dweight=dweight, dbias=dbias)


def _steps(t, name, dtype, shape):
    """Refuses a [batch, L, Dm] operand of another type, shape or channel stride: returns its two strides."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    stride = t.stride()
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the last axis must have stride 1")
    return stride[0], stride[1]


def ss_conv1d_bwd(dout, x, weight, bias=None, window_in=None, dwindow_out=None, silu=True, dx=None, stream=None):
    """Gradients of ss_conv1d (ss_conv1d_bwd): dout [batch, L, Dm] the gradient of its output, the other
    arguments as in the forward call; dwindow_out [batch, Dm, 3] float32 the gradient of window_out or None.

    Returns a dict: dx [batch, L, Dm] (io dtype), dweight [Dm, 4], dbias [Dm] and, with a window_in,
    dwindow_in [batch, Dm, 3] (None without), float32."""
    torch = _load()
    _cuda(x, "x")
    batch, L, Dm = shape = x.shape
    io, f32, dev = x.dtype, torch.float32, x.device
    if dx is None:
        dx = _empty(shape, io, dev, stream)
    s = _ss.ConvGradStrides(_io(io), *_steps(dout, "dout", io, shape), *_steps(x, "x", io, shape), *_steps(dx, "dx", io, shape))
    _param(weight, "weight", f32, (Dm, 4))
    _param(bias, "bias", f32, (Dm,))
    _param(window_in, "window_in", f32, (batch, Dm, 3))
    _param(dwindow_out, "dwindow_out", f32, (batch, Dm, 3))
    dweight, dbias = _empty((Dm, 4), f32, dev, stream), _empty((Dm,), f32, dev, stream)
    dwin = None if window_in is None else _empty((batch, Dm, 3), f32, dev, stream)
    ws, nbytes = _scratch(x, stream, "ss_conv1d_bwd_workspace_size", batch, L, Dm)
    p = _ss._ptr
    st = _ss.lib().ss_conv1d_bwd(dout.data_ptr(), x.data_ptr(), weight.data_ptr(), p(bias), p(window_in), p(dwindow_out), dx.data_ptr(),
                                 dweight.data_ptr(), dbias.data_ptr(), p(dwin), batch, L, Dm, int(bool(silu)), ctypes.byref(s),
                                 ws.data_ptr(), nbytes, _stream(x, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_conv1d_bwd")
    return dict(dx=dx, dweight=dweight, dbias=dbias, dwindow_in=dwin)


def _distill_args(logits, ids, teacher, stream):
    torch = _load()
    _cuda(logits, "logits")
    rows, V = shape = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must be [rows, K]")
    K = ids.shape[1]
    s = _ss.DistillStrides(_io(logits.dtype), _io(teacher.dtype), _rows(logits, "logits", logits.dtype, shape),
                           _rows(ids, "ids", torch.int32, (rows, K)), _rows(teacher, "teacher", teacher.dtype, (rows, K)), V, 1)
    return rows, V, K, s, _empty((rows,), torch.float32, logits.device, stream)


def ss_distill(logits, ids, teacher, temperature=1.0, stream=None):
    """Divergence of the softmax of logits from the teacher's over its top logits, per row (ss_distill).

    logits [rows, V] float32 or bfloat16; ids [rows, K] int32 the columns of the teacher's logits (negative:
    no entry), teacher [rows, K] float32 or bfloat16.  Returns loss [rows] float32."""
    rows, V, K, s, loss = _distill_args(logits, ids, teacher, stream)
    st = _ss.lib().ss_distill(logits.data_ptr(), ids.data_ptr(), teacher.data_ptr(), loss.data_ptr(), rows, V, K, temperature,
                              ctypes.byref(s), _stream(logits, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_distill")
    return loss


def ss_distill_grad(dloss, logits, ids, teacher, temperature=1.0, dlogits=None, stream=None):
    """ss_distill and the gradient of the logits for given gradients of the losses (ss_distill_grad).

    dloss [rows] float32 (any stride, so an expanded value too).  Returns (loss, dlogits): dlogits like
    logits (it may be logits itself)."""
    rows, V, K, s, loss = _distill_args(logits, ids, teacher, stream)
    if dloss.dtype is not _load().float32:
        raise TypeError(f"dloss must be float32, got {dloss.dtype}")
    if dloss.shape != (rows,):
        raise ValueError(f"dloss must have shape ({rows},), got {tuple(dloss.shape)}")
    s.dloss_r = dloss.stride(0)
    if dlogits is None:
        dlogits = _empty((rows, V), logits.dtype, logits.device, stream)
    else:
        s.dlogits_r = _rows(dlogits, "dlogits", logits.dtype, logits.shape)
    st = _ss.lib().ss_distill_grad(dloss.data_ptr(), logits.data_ptr(), ids.data_ptr(), teacher.data_ptr(), loss.data_ptr(),
                                   dlogits.data_ptr(), rows, V, K, temperature, ctypes.byref(s), _stream(logits, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_distill_grad")
    return loss, dlogits


def _xent_args(hidden, weight, targets):
    torch = _load()
    _cuda(hidden, "hidden")
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden must be [tokens, D] and weight [V, D]")
    T, D = hidden.shape
    V = weight.shape[0]
    io = hidden.dtype
    s = _ss.XentStrides(_io(io), _rows(hidden, "hidden", io, (T, D)), _rows(weight, "weight", io, (V, D)), D, D, 1)
    _param(targets, "targets", torch.int32, (T,))
    return T, V, D, s


def ss_linear_xent(hidden, weight, targets, stream=None):
    """Softmax cross entropy over the vocabulary from the last layer's rows (ss_linear_xent): the logits
    hidden @ weight.T are not kept.

    hidden [tokens, D], weight [V, D] (float32 or bfloat16, the same); targets [tokens] int32, negative for a
    row without one.  Returns (loss, lse), both [tokens] float32 and zero in rows without a target; lse is for
    ss_linear_xent_bwd."""
    T, V, D, s = _xent_args(hidden, weight, targets)
    f32, dev = _load().float32, hidden.device
    loss, lse = _empty((T,), f32, dev, stream), _empty((T,), f32, dev, stream)
    ws, nbytes = _scratch(hidden, stream, "ss_linear_xent_workspace_size", T, V, D, s.io_dtype, 0)
    st = _ss.lib().ss_linear_xent(hidden.data_ptr(), weight.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr(), T, V, D,
                                  ctypes.byref(s), ws.data_ptr(), nbytes, _stream(hidden, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_linear_xent")
    return loss, lse


def ss_linear_xent_bwd(dloss, hidden, weight, targets, lse, stream=None):
    """Gradients of ss_linear_xent for given gradients of the losses (ss_linear_xent_bwd): dloss [tokens]
    float32 (any stride, so an expanded value too), lse from the forward call.

    Returns a dict: dhidden like hidden and dweight like weight."""
    T, V, D, s = _xent_args(hidden, weight, targets)
    f32, io, dev = _load().float32, hidden.dtype, hidden.device
    if dloss.dtype is not f32:
        raise TypeError(f"dloss must be float32, got {dloss.dtype}")
    if dloss.shape != (T,):
        raise ValueError(f"dloss must have shape ({T},), got {tuple(dloss.shape)}")
    s.dloss_t = dloss.stride(0)
    _param(lse, "lse", f32, (T,))
    dhidden, dweight = _empty((T, D), io, dev, stream), _empty((V, D), io, dev, stream)
    ws, nbytes = _scratch(hidden, stream, "ss_linear_xent_workspace_size", T, V, D, s.io_dtype, 1)
    st = _ss.lib().ss_linear_xent_bwd(dloss.data_ptr(), hidden.data_ptr(), weight.data_ptr(), targets.data_ptr(), lse.data_ptr(),
                                      dhidden.data_ptr(), dweight.data_ptr(), T, V, D, ctypes.byref(s), ws.data_ptr(), nbytes,
                                      _stream(hidden, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_linear_xent_bwd")
    return dict(dhidden=dhidden, dweight=dweight)
