"""Python binding of the calls that serve a stack of multi-head state space layers: the scan with
its convolution for packed prompts and for single tokens, the residual norm and the sampler.

Argument marshalling only, as in the package's other calls; ``include/selscan.h`` has the
definitions.
"""
from __future__ import annotations

import ctypes

import selective_state_space_scan_gb300 as _ss

_HEADS_WS = {}


def _tensor(t, name, shape=None, dtype=None, contiguous=False, device=None):
    """Refuses what the C call cannot see: types, shapes, layouts and devices of tensors."""
    if t is None:
        return
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor" + ("" if device is None else f" on {device}"))
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not contiguous:
        _ss._check_inner(t, name)


def _empty(shape, dtype, device, stream):
    """An output allocated on the stream that the call runs on, so that its memory is not handed to
    another stream's work while the call may still write it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _row_stride(t):
    return 0 if t is None else t.stride(0)


def _heads_args(xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, y, ints, stream):
    import torch
    io = _ss._io_code(xbc.dtype)
    dev, f32 = xbc.device, torch.float32
    if state.dim() != 4:
        raise ValueError("state must be [slots, H, P, N]")
    n_slots, H, P, N = state.shape
    T, C = xbc.shape
    bc = C - H * P
    if bc <= 0 or bc % (2 * N):
        raise ValueError(f"xbc has {C} channels: H*P + 2*G*N are wanted (H, P, N = {H}, {P}, {N})")
    G = bc // (2 * N)
    if y is None:
        y = _empty((T, H * P), xbc.dtype, dev, stream)
    _tensor(xbc, "xbc")
    _tensor(dt_raw, "dt_raw", (T, H), xbc.dtype, device=dev)
    _tensor(z, "z", (T, H * P), xbc.dtype, device=dev)
    _tensor(y, "y", (T, H * P), xbc.dtype, device=dev)
    _tensor(conv_w, "conv_w", (C, 4), f32, True, dev)
    _tensor(conv_b, "conv_b", (C,), f32, True, dev)
    _tensor(dt_bias, "dt_bias", (H,), f32, True, dev)
    _tensor(A_log, "A_log", (H,), f32, True, dev)
    _tensor(D, "D", (H,), f32, True, dev)
    _tensor(state, "state", None, f32, True, dev)
    _tensor(window, "window", (n_slots, C, 3), f32, True, dev)
    for name, t, n in ints:
        _tensor(t, name, (n,), torch.int32, True, dev)
    s = _ss.HeadsStrides(io, _row_stride(xbc), _row_stride(dt_raw), _row_stride(z), _row_stride(y))
    return io, y, T, H, P, G, N, n_slots, s


def ss_heads_fwd(xbc, dt_raw, conv_w, A_log, state, window, cu_seqlens, conv_b=None, dt_bias=None, D=None, z=None,
                 slots=None, fresh=None, y=None, stream=None):
    """Multi-head selective scan with its causal convolution over packed prompts (ss_heads_fwd).

    xbc [tokens, H*P + 2*G*N], dt_raw [tokens, H], z [tokens, H*P] (float32 or bfloat16, channel
    stride 1, any token stride); conv_w [C, 4], conv_b [C], dt_bias, A_log, D [H] float32.
    state [slots, H, P, N] and window [slots, C, 3] (float32) are the caches, updated in place.
    cu_seqlens [n+1] int32: sequence i is rows cu_seqlens[i] to cu_seqlens[i+1]; slots [n] int32 (None:
    slot i; negative: no slot); fresh [n] int32: non-zero starts from zeros.  Returns y [tokens, H*P]."""
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [sequences + 1]")
    n = cu_seqlens.shape[0] - 1
    io, y, T, H, P, G, N, n_slots, s = _heads_args(
        xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, y,
        (("cu_seqlens", cu_seqlens, n + 1), ("slots", slots, n), ("fresh", fresh, n)), stream)
    key = (n, T, H, P, G, N, io)
    nbytes = _HEADS_WS.get(key)
    if nbytes is None:
        nbytes = _HEADS_WS[key] = int(_ss.lib().ss_heads_workspace_size(*key))
    ws = _ss.workspace_for(xbc.device, stream, nbytes, purpose="heads") if nbytes else None
    p = _ss._ptr
    st = _ss.lib().ss_heads_fwd(p(xbc), p(dt_raw), p(z), p(conv_w), p(conv_b), p(dt_bias), p(A_log), p(D), p(y), p(state),
                                p(window), p(cu_seqlens), p(slots), p(fresh), n, T, H, P, G, N, n_slots, ctypes.byref(s),
                                p(ws), 0 if ws is None else ws.numel(), _ss._stream_handle(stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_heads_fwd")
    return y


def ss_heads_step(state, window, xbc, dt_raw, conv_w, A_log, conv_b=None, dt_bias=None, D=None, z=None, slots=None, y=None,
                  stream=None):
    """One token of every request (ss_heads_step): ss_heads_fwd's tensors with one row per request;
    slots [batch] int32 (None: slot b; negative: a padded row).  Updates state and window in place
    and returns y [batch, H*P]."""
    n = xbc.shape[0]
    io, y, T, H, P, G, N, n_slots, s = _heads_args(xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, y,
                                                   (("slots", slots, n),), stream)
    nbytes = _HEADS_WS.get((n, G))
    if nbytes is None:
        nbytes = _HEADS_WS[n, G] = int(_ss.lib().ss_heads_step_workspace_size(n, G))
    ws = _ss.workspace_for(xbc.device, stream, nbytes, purpose="heads") if nbytes else None
    p = _ss._ptr
    st = _ss.lib().ss_heads_step(p(state), p(window), p(xbc), p(dt_raw), p(z), p(conv_w), p(conv_b), p(dt_bias), p(A_log),
                                 p(D), p(y), p(slots), n, H, P, G, N, n_slots, ctypes.byref(s), p(ws),
                                 0 if ws is None else ws.numel(), _ss._stream_handle(stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_heads_step")
    return y


def _norm_args(x, weight, residual, residual_out, stream):
    import torch
    rows, D = x.shape
    io = _ss._io_code(x.dtype)
    rdt = x.dtype if residual is None else residual.dtype
    res = _ss._io_code(rdt)
    if residual_out is None:
        residual_out = _empty((rows, D), rdt, x.device, stream)
    _tensor(x, "x")
    _tensor(weight, "weight", (D,), torch.float32, True, x.device)
    _tensor(residual, "residual", (rows, D), rdt, device=x.device)
    _tensor(residual_out, "residual_out", (rows, D), rdt, device=x.device)
    return rows, D, io, res, residual_out


def ss_add_rmsnorm(x, weight, residual=None, eps=1e-5, y=None, residual_out=None, stream=None):
    """r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight over rows (ss_add_rmsnorm).

    x [rows, D] and residual [rows, D]: float32 or bfloat16, each its own; weight [D] float32.
    Returns (y, residual_out): y like x, r in the residual's type (residual_out may be residual)."""
    import torch
    rows, D, io, res, residual_out = _norm_args(x, weight, residual, residual_out, stream)
    if y is None:
        y = _empty((rows, D), x.dtype, x.device, stream)
    _tensor(y, "y", (rows, D), x.dtype, device=x.device)
    s = _ss.NormStrides(io, res, x.stride(0), _row_stride(residual), residual_out.stride(0), y.stride(0))
    p = _ss._ptr
    st = _ss.lib().ss_add_rmsnorm(p(x), p(residual), p(weight), p(residual_out), p(y), rows, D, eps, ctypes.byref(s),
                                  _ss._stream_handle(stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_add_rmsnorm")
    return y, residual_out


def ss_add_rmsnorm_f8(x, weight, residual=None, eps=1e-5, block=0, y=None, scale=None, residual_out=None, stream=None):
    """ss_add_rmsnorm with y in float8_e4m3fn and one float32 scale per `block` columns (0: per row).

    Returns (y, residual_out, scale): y[r, c] * scale[r, c // block] stands for the norm's output;
    scale is [rows, ceil(D / block)]."""
    import torch
    rows, D, io, res, residual_out = _norm_args(x, weight, residual, residual_out, stream)
    f8 = torch.float8_e4m3fn
    if y is None:
        y = _empty((rows, D), f8, x.device, stream)
    nb = -(-D // block) if block else 1
    if scale is None:
        scale = _empty((rows, nb), torch.float32, x.device, stream)
    _tensor(y, "y", (rows, D), f8, device=x.device)
    _tensor(scale, "scale", (rows, nb), torch.float32, True, x.device)
    s = _ss.NormStrides(io, res, x.stride(0), _row_stride(residual), residual_out.stride(0), y.stride(0))
    p = _ss._ptr
    st = _ss.lib().ss_add_rmsnorm_f8(p(x), p(residual), p(weight), p(residual_out), p(y), p(scale), rows, D, block, eps,
                                     ctypes.byref(s), _ss._stream_handle(stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_add_rmsnorm_f8")
    return y, residual_out, scale


def ss_sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, stream=None):
    """The next token of every row (ss_sample): temperature, top-k, top-p and min-p, then the argmax of
    weight / noise over what stays.

    logits [rows, V] float32 or bfloat16; noise [rows, V] float32 draws of the exponential distribution;
    temperature, top_p, min_p [rows] float32 and top_k [rows] int32, each None for off.  Returns
    tokens [rows] int32 (-1 for a row without a finite logit)."""
    import torch
    rows, V = logits.shape
    io, dev, f32 = _ss._io_code(logits.dtype), logits.device, torch.float32
    if tokens is None:
        tokens = _empty((rows,), torch.int32, dev, stream)
    _tensor(logits, "logits")
    _tensor(noise, "noise", (rows, V), f32, device=dev)
    _tensor(temperature, "temperature", (rows,), f32, True, dev)
    _tensor(top_k, "top_k", (rows,), torch.int32, True, dev)
    _tensor(top_p, "top_p", (rows,), f32, True, dev)
    _tensor(min_p, "min_p", (rows,), f32, True, dev)
    _tensor(tokens, "tokens", (rows,), torch.int32, True, dev)
    p = _ss._ptr
    st = _ss.lib().ss_sample(p(logits), p(noise), p(temperature), p(top_k), p(top_p), p(min_p), p(tokens), rows, V, io,
                             logits.stride(0), noise.stride(0), _ss._stream_handle(stream))
    if st != 0:
        raise _ss.SelscanError(st, "ss_sample")
    return tokens
