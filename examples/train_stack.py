"""Training a small stack of selective scan layers on the framework's calls: every layer is residual layer norm ->
projection -> convolution -> scan -> projection, the loss is cross entropy over the vocabulary (and, with a
teacher's top logits, distillation from them).  The gradients are written out call by call; the projections are
plain matrix products.

    python examples/train_stack.py            # ten steps on random tokens
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_scan_gb300 as ss  # noqa: E402


class Layer:
    def __init__(self, g, width, Dm, N, R, dtype):
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
        ru = lambda *s: torch.rand(*s, generator=g, device="cuda")           # noqa: E731
        self.Dm, self.N, self.R = Dm, N, R
        self.p = dict(norm_w=1 + 0.1 * rn(width), norm_b=0.1 * rn(width), w_in=(rn(2 * Dm, width) / width ** 0.5).to(dtype),
                      conv_w=0.5 * rn(Dm, 4), conv_b=0.1 * rn(Dm), w_x=(rn(R + 2 * N, Dm) / Dm ** 0.5).to(dtype),
                      w_dt=(rn(Dm, R) / R ** 0.5).to(dtype), dt_bias=-2 - ru(Dm), A_log=torch.log(1 + 7 * ru(Dm, N)), D=1 + 0.1 * rn(Dm),
                      w_out=(rn(width, Dm) / Dm ** 0.5).to(dtype))

    def forward(self, x, residual, batch, L):
        """x and residual [batch * L, width].  Returns (output, new residual, what the backward pass reads)."""
        p, Dm, N, R = self.p, self.Dm, self.N, self.R
        h, r, mean, rstd = ss.ss_add_layernorm(x, p["norm_w"], bias=p["norm_b"], residual=residual)
        uz = (h @ p["w_in"].t()).view(batch, L, 2 * Dm)
        v, z = uz[..., :Dm], uz[..., Dm:]
        u = ss.ss_conv1d(v, p["conv_w"], p["conv_b"], silu=True)
        xp = u @ p["w_x"].t()
        low, B, C = xp[..., :R], xp[..., R:R + N], xp[..., R + N:]
        delta = low @ p["w_dt"].t()
        y, ckpt = ss.ss_fwd_ckpt(u, delta, p["dt_bias"], p["A_log"], B, C, p["D"], z)
        out = y.view(batch * L, Dm) @ p["w_out"].t()
        return out, r, (h, r, mean, rstd, v, z, u, low, B, C, delta, y, ckpt)

    def backward(self, dout, dr, saved):
        """dout the gradient of the output, dr that of the new residual.  Returns (dx, dresidual, parameters')."""
        p, Dm = self.p, self.Dm
        h, r, mean, rstd, v, z, u, low, B, C, delta, y, ckpt = saved
        batch, L, _ = u.shape
        rows = lambda t: t.reshape(batch * L, -1)                            # noqa: E731
        g = ss.ss_bwd((dout @ p["w_out"]).view(batch, L, Dm), u, delta, p["dt_bias"], p["A_log"], B, C, p["D"], z, ckpt=ckpt)
        ddelta = rows(g["ddelta_raw"])
        dxp = torch.cat([ddelta @ p["w_dt"], rows(g["dB"]).to(u.dtype), rows(g["dC"]).to(u.dtype)], 1)
        du = rows(g["du"]) + dxp @ p["w_x"]
        c = ss.ss_conv1d_bwd(du.view(batch, L, Dm), v, p["conv_w"], bias=p["conv_b"], silu=True)
        duz = torch.cat([rows(c["dx"]), rows(g["dz"])], 1)
        n = ss.ss_add_layernorm_bwd(duz @ p["w_in"], r, p["norm_w"], mean, rstd, dr=dr)
        return n["dx"], n["dresidual"], dict(norm_w=n["dweight"], norm_b=n["dbias"], w_in=duz.t() @ h, conv_w=c["dweight"], conv_b=c["dbias"],
                                             w_x=dxp.t() @ rows(u), w_dt=ddelta.t() @ rows(low), dt_bias=g["ddelta_bias"], A_log=g["dA_log"],
                                             D=g["dD"], w_out=dout.t() @ rows(y))


class Model:
    def __init__(self, layers=2, width=64, Dm=128, N=16, R=8, vocab=500, dtype=torch.float32, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
        self.layers = [Layer(g, width, Dm, N, R, dtype) for _ in range(layers)]
        self.p = dict(table=rn(vocab, width).to(dtype), norm_w=torch.ones(width, device="cuda"), norm_b=torch.zeros(width, device="cuda"),
                      head=(rn(vocab, width) / width ** 0.5).to(dtype))

    def step(self, tokens, targets, teacher=None, weight=0.5, temperature=2.0):
        """Mean loss over the targets (negative: none) and its gradients: a list of dicts, the layers' and, last, the
        model's own.  teacher: (ids, logits) [batch * L, K] of a teacher's top logits: `weight` of the loss is then
        the divergence from them."""
        batch, L = tokens.shape
        flat, targets = tokens.reshape(-1).long(), targets.reshape(-1)
        p = self.p
        x = p["table"][flat]
        r, saved = torch.zeros(x.shape, device="cuda"), []
        for layer in self.layers:
            x, r, s = layer.forward(x, r, batch, L)
            saved.append(s)
        h, r, mean, rstd = ss.ss_add_layernorm(x, p["norm_w"], bias=p["norm_b"], residual=r)
        loss, lse = ss.ss_linear_xent(h, p["head"], targets)
        share = 1.0 if teacher is None else 1.0 - weight
        scale = 1.0 / max(1, int((targets >= 0).sum()))
        d = ss.ss_linear_xent_bwd(torch.full((1,), share * scale, device="cuda").expand(batch * L), h, p["head"], targets, lse)
        total = share * scale * loss.sum()
        dh, dhead = d["dhidden"], d["dweight"]
        if teacher is not None:
            ids, top = teacher
            logits = h @ p["head"].t()
            g = torch.full((1,), weight / (batch * L), device="cuda").expand(batch * L)
            kl, dl = ss.ss_distill_grad(g, logits, ids, top, temperature=temperature, dlogits=logits)
            total = total + weight / (batch * L) * kl.sum()
            dh, dhead = dh + dl @ p["head"], dhead + dl.t() @ h
        n = ss.ss_add_layernorm_bwd(dh, r, p["norm_w"], mean, rstd)
        dx, dr = n["dx"], n["dresidual"]
        grads = [dict(norm_w=n["dweight"], norm_b=n["dbias"], head=dhead)]
        for layer, s in zip(self.layers[::-1], saved[::-1]):
            dx, dr, g = layer.backward(dx, dr, s)
            grads.insert(0, g)
        grads[-1]["table"] = torch.zeros_like(p["table"]).index_add_(0, flat, dx)
        return total, grads

    def descend(self, grads, rate):
        for params, g in zip([layer.p for layer in self.layers] + [self.p], grads):
            for k, v in g.items():
                params[k] -= (rate * v).to(params[k].dtype)


def main():
    model = Model()
    g = torch.Generator("cuda").manual_seed(1)
    tokens = torch.randint(0, 500, (4, 65), generator=g, device="cuda", dtype=torch.int32)
    for i in range(10):
        loss, grads = model.step(tokens[:, :-1], tokens[:, 1:])
        model.descend(grads, 0.5)
        print(f"step {i}: loss {float(loss):.4f}")
    assert ss.device_error() == 0


if __name__ == "__main__":
    main()
