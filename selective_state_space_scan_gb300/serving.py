"""Python binding of the calls that serve a stack of multi-head state space layers: the scan with
its convolution for packed prompts and for single tokens, the residual norm and the sampler.

Argument marshalling only, as in the package's other calls; ``include/selscan.h`` has the
definitions.
"""
from __future__ import annotations

import ctypes

import selective_state_space_scan_gb300 as _ss

_HEADS_BYTES = {}
_HEADS_WS = {}
_IO = {}
_torch = None
_lib = None


def _load():
    """The torch module and the library, looked up once: the calls below are made once per layer and
    token, where a few microseconds of marshalling are as long as the kernels."""
    global _torch, _lib
    if _torch is None:
        import torch
        _lib = _ss.lib()
        _IO.update({torch.float32: _ss.SS_F32, torch.bfloat16: _ss.SS_BF16})
        _torch = torch
    return _torch


def _io(dtype):
    code = _IO.get(dtype)
    return _ss._io_code(dtype) if code is None else code      # (which refuses other types)


def _stream(t, stream):
    """Handle of the stream that the call runs on."""
    if stream is not None:
        return stream.cuda_stream
    return _torch._C._cuda_getCurrentRawStream(t.get_device())


def _empty(shape, dtype, device, stream):
    """An output allocated on the stream that the call runs on, so that its memory is not handed to
    another stream's work while the call may still write it."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _workspace(t, stream, handle, nbytes):
    """The heads calls' workspace: one buffer per device and stream, zero-filled when it is made (one of its own
    for every capture: see workspace_for)."""
    if _lib.ss__capture_id(handle):
        return _ss.workspace_for(t.device, stream, nbytes, purpose="heads")
    key = (t.get_device(), handle)
    ws = _HEADS_WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _HEADS_WS[key] = _ss.workspace_for(t.device, stream, nbytes, purpose="heads")
    return ws


def _param(t, name, dtype, shape):
    """Refuses a contiguous operand of another type, shape or layout (None passes)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtype, shape):
    """The same for a two-dimensional operand with any row stride: returns the stride (0 for None)."""
    if t is None:
        return 0
    stride = t.stride()
    if t.dtype is dtype and t.shape == shape and (stride[1] == 1 or shape[1] <= 1):
        return stride[0]
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: the last axis must have stride 1")


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _heads_args(xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, y, stream):
    torch = _load()
    _cuda(xbc, "xbc")
    dtype, f32 = xbc.dtype, torch.float32
    if state.dim() != 4 or xbc.dim() != 2:
        raise ValueError("state must be [slots, H, P, N] and xbc [rows, channels]")
    n_slots, H, P, N = state.shape
    T, C = xbc.shape
    HP = H * P
    G, rest = divmod(C - HP, 2 * N) if N else (0, 1)
    if G <= 0 or rest:
        raise ValueError(f"xbc has {C} channels: H*P + 2*G*N are wanted (H, P, N = {H}, {P}, {N})")
    if y is None:
        y = _empty((T, HP), dtype, xbc.device, stream)
    s = _ss.HeadsStrides(_io(dtype), _rows(xbc, "xbc", dtype, (T, C)), _rows(dt_raw, "dt_raw", dtype, (T, H)),
                         _rows(z, "z", dtype, (T, HP)), _rows(y, "y", dtype, (T, HP)))
    _param(conv_w, "conv_w", f32, (C, 4))
    _param(conv_b, "conv_b", f32, (C,))
    _param(dt_bias, "dt_bias", f32, (H,))
    _param(A_log, "A_log", f32, (H,))
    _param(D, "D", f32, (H,))
    _param(state, "state", f32, state.shape)
    _param(window, "window", f32, (n_slots, C, 3))
    return y, T, H, P, G, N, n_slots, s


def ss_heads_fwd(xbc, dt_raw, conv_w, A_log, state, window, cu_seqlens, conv_b=None, dt_bias=None, D=None, z=None,
                 slots=None, fresh=None, y=None, stream=None):
    """Multi-head selective scan with its causal convolution over packed prompts (ss_heads_fwd).

    xbc [tokens, H*P + 2*G*N], dt_raw [tokens, H], z [tokens, H*P] (float32 or bfloat16, channel
    stride 1, any token stride); conv_w [C, 4], conv_b [C], dt_bias, A_log, D [H] float32.
    state [slots, H, P, N] and window [slots, C, 3] (float32) are the caches, updated in place.
    cu_seqlens [n+1] int32: sequence i is rows cu_seqlens[i] to cu_seqlens[i+1]; slots [n] int32 (None:
    slot i; negative: no slot); fresh [n] int32: non-zero starts from zeros.  Returns y [tokens, H*P]."""
    y, T, H, P, G, N, n_slots, s = _heads_args(xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, y, stream)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [sequences + 1]")
    n, i32 = cu_seqlens.shape[0] - 1, _torch.int32
    _param(cu_seqlens, "cu_seqlens", i32, (n + 1,))
    _param(slots, "slots", i32, (n,))
    _param(fresh, "fresh", i32, (n,))
    sizes = (n, T, H, P, G, N, s.io_dtype)
    key = (xbc.get_device(), sizes)                            # (the plan depends on the device's SM count)
    nbytes = _HEADS_BYTES.get(key)
    if nbytes is None:
        nbytes = _ss._remember(_HEADS_BYTES, key, int(_lib.ss_heads_workspace_size(*sizes)))
    handle = _stream(xbc, stream)
    p = _ss._ptr
    with _ss._stream_lock(handle):
        ws = _workspace(xbc, stream, handle, nbytes)
        st = _lib.ss_heads_fwd(xbc.data_ptr(), dt_raw.data_ptr(), p(z), conv_w.data_ptr(), p(conv_b), p(dt_bias),
                               A_log.data_ptr(), p(D), y.data_ptr(), state.data_ptr(), window.data_ptr(), cu_seqlens.data_ptr(),
                               p(slots), p(fresh), n, T, H, P, G, N, n_slots, ctypes.byref(s), ws.data_ptr(), ws.numel(), handle)
    if st != 0:
        raise _ss.SelscanError(st, "ss_heads_fwd")
    return y


def ss_heads_step(state, window, xbc, dt_raw, conv_w, A_log, conv_b=None, dt_bias=None, D=None, z=None, slots=None, y=None,
                  stream=None):
    """One token of every request (ss_heads_step): ss_heads_fwd's tensors with one row per request;
    slots [batch] int32 (None: slot b; negative: a padded row).  Updates state and window in place
    and returns y [batch, H*P]."""
    y, n, H, P, G, N, n_slots, s = _heads_args(xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, y, stream)
    _param(slots, "slots", _torch.int32, (n,))
    key = (n, G)                                               # (the same on every device)
    nbytes = _HEADS_BYTES.get(key)
    if nbytes is None:
        nbytes = _ss._remember(_HEADS_BYTES, key, int(_lib.ss_heads_step_workspace_size(n, G)))
    handle = _stream(xbc, stream)
    p = _ss._ptr
    with _ss._stream_lock(handle):
        ws = _workspace(xbc, stream, handle, nbytes)
        st = _lib.ss_heads_step(state.data_ptr(), window.data_ptr(), xbc.data_ptr(), dt_raw.data_ptr(), p(z), conv_w.data_ptr(),
                                p(conv_b), p(dt_bias), A_log.data_ptr(), p(D), y.data_ptr(), p(slots), n, H, P, G, N, n_slots,
                                ctypes.byref(s), ws.data_ptr(), ws.numel(), handle)
    if st != 0:
        raise _ss.SelscanError(st, "ss_heads_step")
    return y


def _norm_args(x, weight, residual, residual_out, y, ydtype, stream):
    torch = _load()
    _cuda(x, "x")
    rows, D = shape = x.shape
    dtype = x.dtype
    rdt = dtype if residual is None else residual.dtype
    if residual_out is None:
        residual_out = _empty(shape, rdt, x.device, stream)
    if y is None:
        y = _empty(shape, ydtype or dtype, x.device, stream)
    s = _ss.NormStrides(_io(dtype), _io(rdt), _rows(x, "x", dtype, shape),
                        _rows(residual, "residual", rdt, shape), _rows(residual_out, "residual_out", rdt, shape),
                        _rows(y, "y", ydtype or dtype, shape))
    _param(weight, "weight", torch.float32, (D,))
    return rows, D, residual_out, y, s


def ss_add_rmsnorm(x, weight, residual=None, eps=1e-5, y=None, residual_out=None, stream=None):
    """r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight over rows (ss_add_rmsnorm).

    x [rows, D] and residual [rows, D]: float32 or bfloat16, each its own; weight [D] float32.
    Returns (y, residual_out): y like x, r in the residual's type (residual_out may be residual)."""
    rows, D, residual_out, y, s = _norm_args(x, weight, residual, residual_out, y, None, stream)
    st = _lib.ss_add_rmsnorm(x.data_ptr(), _ss._ptr(residual), weight.data_ptr(), residual_out.data_ptr(), y.data_ptr(), rows, D,
                             eps, ctypes.byref(s), _stream(x, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_add_rmsnorm")
    return y, residual_out


def ss_add_rmsnorm_f8(x, weight, residual=None, eps=1e-5, block=0, y=None, scale=None, residual_out=None, stream=None):
    """ss_add_rmsnorm with y in float8_e4m3fn and one float32 scale per `block` columns (0: per row).

    Returns (y, residual_out, scale): y[r, c] * scale[r, c // block] stands for the norm's output;
    scale is [rows, ceil(D / block)]."""
    torch = _load()
    rows, D, residual_out, y, s = _norm_args(x, weight, residual, residual_out, y, torch.float8_e4m3fn, stream)
    nb = -(-D // block) if block > 0 else 1
    if scale is None:
        scale = _empty((rows, nb), torch.float32, x.device, stream)
    else:
        _param(scale, "scale", torch.float32, (rows, nb))
    st = _lib.ss_add_rmsnorm_f8(x.data_ptr(), _ss._ptr(residual), weight.data_ptr(), residual_out.data_ptr(), y.data_ptr(),
                                scale.data_ptr(), rows, D, block, eps, ctypes.byref(s), _stream(x, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_add_rmsnorm_f8")
    return y, residual_out, scale


def ss_sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, stream=None):
    """The next token of every row (ss_sample): temperature, top-k, top-p and min-p, then the argmax of
    weight / noise over what stays.

    logits [rows, V] float32 or bfloat16; noise [rows, V] float32 draws of the exponential distribution;
    temperature, top_p, min_p [rows] float32 and top_k [rows] int32, each None for off.  Returns
    tokens [rows] int32 (-1 for a row without a finite logit)."""
    torch = _load()
    _cuda(logits, "logits")
    shape, dtype, f32, i32 = logits.shape, logits.dtype, torch.float32, torch.int32
    rows, V = shape
    io, per_row = _io(dtype), (rows,)
    if tokens is None:
        tokens = _empty(per_row, i32, logits.device, stream)
    else:
        _param(tokens, "tokens", i32, per_row)
    logits_r, noise_r = _rows(logits, "logits", dtype, shape), _rows(noise, "noise", f32, shape)
    _param(temperature, "temperature", f32, per_row)
    _param(top_k, "top_k", i32, per_row)
    _param(top_p, "top_p", f32, per_row)
    _param(min_p, "min_p", f32, per_row)
    p = _ss._ptr
    st = _lib.ss_sample(logits.data_ptr(), noise.data_ptr(), p(temperature), p(top_k), p(top_p), p(min_p), tokens.data_ptr(),
                        rows, V, io, logits_r, noise_r, _stream(logits, stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_sample")
    return tokens
