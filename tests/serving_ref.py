"""The serving operators' definitions in 64 bits (numpy), for the tests to compare against."""
import numpy as np


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(v, 0.0)


def heads(xbc, dt_raw, conv_w, conv_b, dt_bias, A_log, D, z, state, window, P, N):
    """One sequence: xbc [L, C], dt_raw [L, H], z [L, H*P] or None, state [H, P, N], window [C, 3]; all
    float64.  Returns (y [L, H*P], state, window)."""
    L, C = xbc.shape
    H = A_log.shape[0]
    G = (C - H * P) // (2 * N)
    e = np.concatenate([window.T, xbc], 0)                   # [3 + L, C]
    y = np.zeros((L, H * P))
    S = state.copy()
    b = np.zeros(C) if conv_b is None else conv_b
    tb = np.zeros(H) if dt_bias is None else dt_bias
    Dv = np.zeros(H) if D is None else D
    for t in range(L):
        u = silu(b + sum(conv_w[:, k] * e[t + k] for k in range(4)))
        x = u[:H * P].reshape(H, P)
        B = np.repeat(u[H * P:H * P + G * N].reshape(G, N), H // G, 0)
        Cm = np.repeat(u[H * P + G * N:].reshape(G, N), H // G, 0)
        dt = softplus(dt_raw[t] + tb)
        a = np.exp(-dt * np.exp(A_log))
        S = S * a[:, None, None] + (dt[:, None] * x)[:, :, None] * B[:, None, :]
        y[t] = ((S * Cm[:, None, :]).sum(-1) + Dv[:, None] * x).ravel()
        if z is not None:
            y[t] *= silu(z[t])
    return y, S, e[L:].T.copy()


def norm(x, residual, weight, eps):
    r = x if residual is None else x + residual
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * weight, r


def e4m3_nearest(v):
    """The e4m3 value nearest to each v (ties to even), |v| <= 464."""
    a = np.abs(v)
    with np.errstate(divide="ignore"):
        e = np.clip(np.floor(np.log2(np.where(a > 0, a, 1e-300))), -6, 8)
    step = 2.0 ** (e - 3)
    return np.sign(v) * np.minimum(np.round(a / step) * step, 448.0)


def sample_row(l, noise, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    l = np.minimum(l, np.finfo(np.float32).max)
    order = np.argsort(-l, kind="stable")
    if l[order[0]] == -np.inf:
        return -1
    if temperature <= 0:
        return int(order[0])
    ls = l[order]
    w = np.exp((ls - ls[0]) / temperature)
    k = top_k if 0 < top_k < len(l) else len(l)
    keep = np.arange(len(l)) < k
    total = w[keep].sum()
    excl = np.cumsum(w) - w
    if top_p < 1:
        keep &= excl < top_p * total
    keep &= w >= min_p
    keep[0] = True
    with np.errstate(divide="ignore"):
        key = np.where(keep, w / noise.astype(np.float64)[order], -1.0)
    return int(order[key == key.max()].min())
