"""The training operators' definitions in 64 bits (numpy), for the tests to compare against."""
import numpy as np


def layernorm(x, residual, w, b, eps):
    r = x if residual is None else x + residual
    mean = r.mean(-1)
    rstd = 1.0 / np.sqrt(((r - mean[:, None]) ** 2).mean(-1) + eps)
    y = (r - mean[:, None]) * rstd[:, None] * w + (0.0 if b is None else b)
    return y, r, mean, rstd


def layernorm_bwd(dy, r, w, mean, rstd, dr=None):
    """Returns (d, dweight, dbias), d the gradient of x and of residual."""
    xh = (r - mean[:, None]) * rstd[:, None]
    a = dy * w
    d = rstd[:, None] * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
    return d if dr is None else d + dr, (dy * xh).sum(0), dy.sum(0)


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _samples(x, window):
    batch, L, Dm = x.shape
    win = np.zeros((batch, Dm, 3)) if window is None else window
    return np.concatenate([win.transpose(0, 2, 1), x], 1)                # [batch, 3 + L, Dm]


def conv1d(x, w, b, window, silu):
    """Returns (out, window_out)."""
    e, L = _samples(x, window), x.shape[1]
    v = sum(w[:, k] * e[:, k:k + L] for k in range(4)) + (0.0 if b is None else b)
    return (v * _sigmoid(v) if silu else v), e[:, L:].transpose(0, 2, 1).copy()


def conv1d_bwd(dout, x, w, b, window, dwindow_out, silu):
    """Returns (dx, dweight, dbias, dwindow_in)."""
    e, L = _samples(x, window), x.shape[1]
    g = dout
    if silu:
        v = sum(w[:, k] * e[:, k:k + L] for k in range(4)) + (0.0 if b is None else b)
        s = _sigmoid(v)
        g = dout * s * (1.0 + v * (1.0 - s))
    de = np.zeros_like(e)
    if dwindow_out is not None:
        de[:, L:] += dwindow_out.transpose(0, 2, 1)
    for k in range(4):
        de[:, k:k + L] += w[:, k] * g
    dw = np.stack([(g * e[:, k:k + L]).sum((0, 1)) for k in range(4)], 1)
    return de[:, 3:], dw, g.sum((0, 1)), de[:, :3].transpose(0, 2, 1)


def xent(h, w, t):
    """Returns (loss, lse): zero in rows without a target (t < 0)."""
    l = h @ w.T
    m = l.max(1)
    lse = m + np.log(np.exp(l - m[:, None]).sum(1))
    ok = t >= 0
    return np.where(ok, lse - l[np.arange(len(t)), np.where(ok, t, 0)], 0.0), np.where(ok, lse, 0.0)


def xent_bwd(dloss, h, w, t):
    """Returns (dhidden, dweight); rows without a target count for nothing, whatever they hold."""
    ok = t >= 0
    dh, hv, tv = np.zeros_like(h), h[ok], t[ok]
    l = hv @ w.T
    p = np.exp(l - l.max(1, keepdims=True)) if len(tv) else l
    p = p / p.sum(1, keepdims=True)
    p[np.arange(len(tv)), tv] -= 1.0
    p *= dloss[ok][:, None]
    dh[ok] = p @ w
    return dh, p.T @ hv


def distill(z, ids, teacher, tau, dloss=None):
    """Returns (loss, dlogits)."""
    rows, V = z.shape
    loss, dz = np.zeros(rows), np.zeros((rows, V))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for i in range(rows):
            ok = (ids[i] >= 0) & (ids[i] < V) & (teacher[i] != -np.inf)
            at, t = ids[i][ok], teacher[i][ok] / tau
            if not len(at):
                continue
            lp = t - t.max()
            lp = lp - np.log(np.exp(lp).sum())
            lq = z[i] / tau - z[i].max() / tau
            lq = lq - np.log(np.exp(lq).sum())
            p, q = np.exp(lp), np.exp(lq)
            loss[i] = (p * (lp - lq[at]))[p != 0].sum()
            np.subtract.at(q, at, p)
            if dloss is not None:
                dz[i] = dloss[i] / tau * q
    return loss, dz
