"""Element-wise bounds of the cross entropy's gradients, for tests that look at every row by itself.

With p the softmax in 64 bits, d = (p - [target]) dloss the gradient of the logits and n, m the norms of the rows:
  logits   sums in fp32 of D products (fp32 tensors: six times the additions), each within 2^-23 of the partial sum:
           p is off by q = 4 (D/16 (6) + 16) 2^-23 n m + 2^-20 of itself (the factor 4: logit and lse, each with its own
           exponential's or logarithm's roundings)
  dl       rounded to u of itself: one fp16 2^-11, two bf16 2^-16, two fp16 2^-22; fp16 counts in steps of 2^-24 from a
           scale that puts dloss of the row above 2^14: 2^-39 of |dloss|
  hidden   exact in bf16; in fp32 2^-22 of itself or 2^-38 of the largest; the rows that dweight takes are scaled by dloss
           as well: 2^-38 of the largest value times the largest dloss
  weight   exact in bf16, in fp32 2^-22 of itself, both down to 2^-28 of the largest
  sums     chains of 64 additions cut off at 2^-23 of the partial sum, then rounded ones: 2^-16 of the terms' magnitudes
  result   2^-8 of itself in bf16, 2^-22 in fp32 (sums of slices)"""
import torch

CHUNK = 4096


def _abs_product(a, b):
    """|a| |b| from below 1% above (fp32 is enough for a bound)."""
    return 1.01 * torch.matmul(a.abs().float(), b.abs().float()).double()


def gradients(h, w, t, g, w_kept=2.0 ** -28):
    """The definition in doubles: dict of dhidden, dweight and their bounds (rows without a target: zeros).  w_kept: what
    weights are off by besides, as a part of the largest."""
    T, D = h.shape
    f32 = h.dtype is torch.float32
    u = 2.0 ** -22 if f32 else 2.0 ** -11 if T > 256 else 2.0 ** -16
    own = 2.0 ** -22 if f32 else 2.0 ** -8
    exact = 2.0 ** -22 if f32 else 0.0
    ok = t >= 0
    rows = torch.nonzero(ok)[:, 0]
    hd, wd, gd = h.double(), w.double(), g.double()
    dh, bh = torch.zeros(T, D, dtype=torch.float64, device=h.device), torch.zeros(T, D, dtype=torch.float64, device=h.device)
    dw, bw = torch.zeros_like(wd), torch.zeros_like(wd)
    steps = D / 16 * (6 if f32 else 1) + 16
    q_all = 4 * steps * 2.0 ** -23 * hd.norm(dim=1) * wd.norm(dim=1).max() + 2.0 ** -20
    w_floor = w_kept * float(wd.abs().max())
    x_most, g_most = (float(hd[rows].abs().max()), float(gd[rows].abs().max())) if len(rows) else (0.0, 0.0)
    for i in range(0, len(rows), CHUNK):
        r = rows[i:i + CHUNK]
        x, gr, q = hd[r], gd[r][:, None], q_all[r][:, None]
        p = torch.softmax(x @ wd.t(), 1)
        e = p.clone()
        e[torch.arange(len(r), device=h.device), t[r].long()] -= 1.0
        d = e * gr
        off = (u + exact + 2.0 ** -16) * d.abs() + q * p * gr.abs() + 2.0 ** -39 * gr.abs()      # of dl, and of the sums
        dh[r] = d @ wd
        bh[r] = _abs_product(off, wd) + (w_floor * d.abs().sum(1))[:, None]
        dw += d.t() @ x
        bw += _abs_product(off.t(), x) + 2.0 ** -38 * x_most * g_most * e.abs().sum(0)[:, None]
    return dict(dhidden=dh, dweight=dw, dhidden_bound=bh + own * dh.abs(), dweight_bound=bw + own * dw.abs())


def worst(got, want, k):
    """Largest error of output k, in bounds (a NaN counts as infinitely far)."""
    off = (got[k].double() - want[k]).abs()
    bound = want[k + "_bound"]
    return float(torch.where(off <= bound, torch.where(bound > 0, off / bound, 0.0), torch.where(off.isnan(), float("inf"), off / bound)).max())
