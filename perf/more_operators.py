"""Workloads of the operators that train a stack of state space layers next to its scan.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as the library's
calls, chosen by ``own``:

  norm      residual addition and layer norm, forward and backward, with the gradients of its weight
            and bias
  conv      backward of the causal convolution and SiLU that feed the scan
  xent      softmax cross entropy of the tokens over the vocabulary, from the last layer's rows and
            the output embedding, without keeping the logits; the loss alone or with its gradients
  distill   divergence from a teacher's distribution over its top logits; the loss alone or with the
            gradient of the logits

``listed()`` gives fixed cases, ``draw(rng)`` further ones of the same ranges, ``prepare`` what a
program holds before the call, ``run`` one pass, ``work`` the bytes and operations it cannot do
without, ``exact`` the result in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm of one short sequence in a small model: latency counts
        dict(name="norm of 64 rows", op="norm", rows=64, D=768, io="f32", res="f32", residual=True),
        # an odd width without a residual stream: no wide accesses
        dict(name="norm of odd rows", op="norm", rows=4001, D=1111, io="bf16", res="bf16", residual=False),
        # a training batch of 4 sequences of 8192 tokens, the residual stream in 32 bits: the largest
        dict(name="norm of 32k rows", op="norm", rows=32768, D=2560, io="bf16", res="f32", residual=True),
        # fine-tuning on one short turn that continues from a window
        dict(name="conv of 45 steps", op="conv", batch=1, L=45, Dm=1536, io="bf16", silu=True, window=True),
        # the small model's training batch in 32 bits
        dict(name="conv of 8 x 2048", op="conv", batch=8, L=2048, Dm=1536, io="f32", silu=True, window=False),
        # the large model's training batch
        dict(name="conv of 4 x 8192", op="conv", batch=4, L=8192, Dm=5120, io="bf16", silu=True, window=False),
        # scoring one short text: the output embedding is read for few tokens
        dict(name="loss of 45 tokens", op="xent", tokens=45, D=768, V=50257, io="bf16", ignored=0.0, grad=False),
        # a training step of the small model in 32 bits
        dict(name="step of 2048 tokens", op="xent", tokens=2048, D=768, V=50257, io="f32", ignored=0.0, grad=True),
        # a fine-tuning step on a large vocabulary, the prompts' tokens without a target: the largest call
        dict(name="step of 4096 tokens", op="xent", tokens=4096, D=2048, V=128000, io="bf16", ignored=0.15, grad=True),
        # scoring a long document, an odd number of tokens
        dict(name="loss of 8191 tokens", op="xent", tokens=8191, D=2560, V=50257, io="bf16", ignored=0.0, grad=False),
        # a short answer distilled from a teacher's 16 likeliest tokens
        dict(name="distill 37 tokens", op="distill", rows=37, V=50257, K=16, io="f32", temperature=1.0, empty=0.0, grad=True),
        # a training batch distilled on a large vocabulary, the prompts' tokens without a teacher
        dict(name="distill 4096 tokens", op="distill", rows=4096, V=128000, K=64, io="bf16", temperature=2.0, empty=0.1,
             grad=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "conv", "xent", "xent", "distill"))
    io = rng.choice(("bf16", "bf16", "f32"))
    grad = rng.random() < 0.7
    if op == "norm":
        D = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            D = -(-D // 128) * 128
        rows = _log_int(rng, 1, min(32768, 32768 * 2560 // D))
        residual = rng.random() < 0.7
        return dict(op=op, rows=rows, D=D, io=io, res=rng.choice(("f32", io)) if residual else io, residual=residual)
    if op == "conv":
        Dm = _log_int(rng, 32, 5120)
        if rng.random() < 0.7:
            Dm = -(-Dm // 32) * 32
        batch = rng.randint(1, 8)
        return dict(op=op, batch=batch, L=_log_int(rng, 1, 32768 // batch), Dm=Dm, io=io, silu=rng.random() < 0.8,
                    window=rng.random() < 0.4)
    V = _log_int(rng, 1000, 128000)
    if op == "xent":
        D = _log_int(rng, 64, 2560)
        if rng.random() < 0.7:
            D = -(-D // 64) * 64
        # 32 bits cost more: fewer tokens there
        most = 4096 * 2048 * 128000 // (D * V * (8 if io == "f32" else 1))
        return dict(op=op, tokens=_log_int(rng, 1, min(8192, most)), D=D, V=V, io=io, ignored=rng.choice((0.0, 0.15, 0.5)),
                    grad=grad)
    rows = _log_int(rng, 1, 2048 if io == "f32" else 4096)
    return dict(op=op, rows=rows, V=V, K=_log_int(rng, 1, 128), io=io, temperature=rng.choice((1.0, 2.0, 4.0)),
                empty=rng.choice((0.0, 0.1, 0.4)), grad=grad)


def _trained(case):
    """Rows that have a target (or a teacher): the others have a loss and gradients of zero."""
    n = case["tokens"] if case["op"] == "xent" else case["rows"]
    return n - int(n * case["ignored" if case["op"] == "xent" else "empty"])


# ----------------------------------------------------------------------------------- the inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _by_rows(f, rows, width):
    """f(rows of one part) for all rows, part by part: the draws need not lie in memory in 32 bits at once."""
    step = max(1, (1 << 28) // max(1, width))
    return torch.cat([f(min(step, rows - i)) for i in range(0, rows, step)])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed) % (1 << 62))
    rn = lambda *sh: torch.randn(*sh, generator=g, device="cuda")        # noqa: E731
    ru = lambda *sh: torch.rand(*sh, generator=g, device="cuda")         # noqa: E731
    op, io, s = case["op"], _dtype(case["io"]), dict(case=case)
    if op == "norm":
        rows, D, res = case["rows"], case["D"], _dtype(case["res"])
        s.update(x=(0.3 + rn(rows, D)).to(io), weight=1.0 + 0.2 * rn(D), bias=0.1 * rn(D), dy=rn(rows, D).to(io),
                 residual=(3.0 * rn(rows, D)).to(res) if case["residual"] else None,
                 dr=rn(rows, D).to(res) if case["residual"] else None)
        return s
    if op == "conv":
        b, L, Dm = case["batch"], case["L"], case["Dm"]
        s.update(x=rn(b, L, Dm).to(io), weight=0.5 * rn(Dm, 4), bias=0.1 * rn(Dm), dout=rn(b, L, Dm).to(io),
                 window=rn(b, Dm, 3) if case["window"] else None)
        return s
    if op == "xent":
        T, D, V = case["tokens"], case["D"], case["V"]
        weight = _by_rows(lambda n: (1.5 / D ** 0.5 * rn(n, D)).to(io), V, D)
        targets = torch.randint(V, (T,), generator=g, device="cuda")
        # rows that point toward their target's embedding, as a trained model's do
        hidden = (rn(T, D) + 3.0 * weight[targets].float()).to(io)
        without = torch.randperm(T, generator=g, device="cuda")[_trained(case):]
        targets = targets.to(torch.int32)
        targets[without] = -1
        s.update(hidden=hidden, weight=weight, targets=targets, dloss=torch.full((T,), 1.0 / max(1, _trained(case)), device="cuda"))
        return s
    rows, V, K = case["rows"], case["V"], case["K"]
    logits = _by_rows(lambda n: (2.5 * rn(n, V)).to(io), rows, V)
    # the teacher: the student's logits, off by some noise; its K largest, in decreasing order
    step = max(1, (1 << 27) // V)
    top = [torch.topk(part.float() + rn(part.shape[0], V), K) for part in logits.split(step)]
    teacher, ids = torch.cat([t.values for t in top]), torch.cat([t.indices for t in top])
    # some rows have fewer entries, some none
    have = torch.where(ru(rows) < 0.2, 1 + (ru(rows) * K).long().clamp(max=K - 1), K)
    have[torch.randperm(rows, generator=g, device="cuda")[_trained(case):]] = 0
    ids = torch.where(torch.arange(K, device="cuda")[None] < have[:, None], ids, -1).to(torch.int32)
    s.update(logits=logits, ids=ids, teacher=teacher, dloss=torch.full((rows,), 1.0 / max(1, _trained(case)), device="cuda"))
    return s


# -------------------------------------------------------------------------------- the plain forms

def _plain_norm(s):
    io = s["x"].dtype
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    D = r.shape[1]
    mean = r.sum(-1, keepdim=True) / D
    c = r - mean
    rstd = torch.rsqrt((c * c).sum(-1, keepdim=True) / D + EPS)
    xh = c * rstd
    out = dict(y=(xh * s["weight"] + s["bias"]).to(io), mean=mean[:, 0], rstd=rstd[:, 0])
    if s["residual"] is not None:
        # the backward pass reads the stored sum
        out["residual"] = r.to(s["residual"].dtype)
        xh = (out["residual"].float() - mean) * rstd
    dy = s["dy"].float()
    wdy = dy * s["weight"]
    d = (wdy - wdy.sum(-1, keepdim=True) / D - xh * ((wdy * xh).sum(-1, keepdim=True) / D)) * rstd
    if s["dr"] is not None:
        d = d + s["dr"].float()
        out["dresidual"] = d.to(s["dr"].dtype)
    # (sums over many rows in 64 bits)
    out.update(dx=d.to(io), dweight=(dy * xh).sum(0, dtype=torch.float64).float(), dbias=dy.sum(0, dtype=torch.float64).float())
    return out


def _plain_conv(s):
    x, w, L = s["x"].float(), s["weight"], s["x"].shape[1]
    first = torch.zeros_like(x[:, :1]).expand(-1, 3, -1) if s["window"] is None else s["window"].transpose(1, 2)
    e = torch.cat([first, x], 1)
    g = s["dout"].float()
    if s["case"]["silu"]:
        v = s["bias"] + w[:, 0] * e[:, 0:L] + w[:, 1] * e[:, 1:L + 1] + w[:, 2] * e[:, 2:L + 2] + w[:, 3] * e[:, 3:L + 3]
        sig = 1.0 / (1.0 + torch.exp(-v))
        g = g * (sig * (1.0 + v * (1.0 - sig)))
        del v, sig
    de = torch.zeros_like(e)
    for k in range(4):
        de[:, k:k + L] += w[:, k] * g
    # (sums over many steps in 64 bits)
    dw = torch.stack([(g * e[:, k:k + L]).sum((0, 1), dtype=torch.float64) for k in range(4)], 1)
    out = dict(dx=de[:, 3:].to(s["x"].dtype), dweight=dw.float(), dbias=g.sum((0, 1), dtype=torch.float64).float())
    if s["window"] is not None:
        out["dwindow_in"] = de[:, :3].transpose(1, 2).contiguous()
    return out


def _plain_xent(s):
    h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"].long()
    valid = t >= 0
    at = torch.where(valid, t, 0)[:, None]
    l = torch.matmul(h, w.t())
    m = l.amax(-1, keepdim=True)
    lt = torch.gather(l, 1, at)[:, 0]
    l = torch.exp(l - m)
    total = l.sum(-1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    out = dict(loss=torch.where(valid, lse - lt, 0.0), lse=torch.where(valid, lse, 0.0))
    if s["case"]["grad"]:
        l = l / total
        l.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        l = l * torch.where(valid, s["dloss"], 0.0)[:, None]
        out.update(dhidden=torch.matmul(l, w).to(s["hidden"].dtype), dweight=torch.matmul(l.t(), h).to(s["weight"].dtype))
    return out


def _plain_distill(s):
    z, ids, T = s["logits"].float(), s["ids"].long(), s["case"]["temperature"]
    have = ids >= 0
    t = torch.where(have, s["teacher"], -math.inf)
    mt = torch.clamp(t.amax(-1, keepdim=True), min=-1e30)
    p = torch.where(have, torch.exp((t - mt) / T), 0.0)
    pt = p.sum(-1, keepdim=True)
    row = pt[:, 0] > 0
    p = p / torch.where(pt > 0, pt, 1.0)
    m = z.amax(-1, keepdim=True)
    zi = torch.gather(z, 1, torch.where(have, ids, 0))
    z = torch.exp((z - m) / T)
    total = z.sum(-1, keepdim=True)
    lq = (zi - m) / T - torch.log(total)
    lp = (t - mt) / T - torch.log(torch.where(pt > 0, pt, 1.0))
    out = dict(loss=torch.where(p > 0, p * (lp - lq), 0.0).sum(-1))
    if s["case"]["grad"]:
        g = torch.where(row, s["dloss"], 0.0)[:, None] / T
        z = z / total
        z.scatter_add_(1, torch.where(have, ids, 0), -p)
        out["dlogits"] = (z * g).to(s["logits"].dtype)
    return out


def run(s):
    op, c = s["case"]["op"], s["case"]
    if not own:
        return dict(norm=_plain_norm, conv=_plain_conv, xent=_plain_xent, distill=_plain_distill)[op](s)
    import selective_state_space_scan_gb300 as ss
    if op == "norm":
        y, r, mean, rstd = ss.ss_add_layernorm(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], eps=EPS)
        out = dict(y=y, mean=mean, rstd=rstd)
        g = ss.ss_add_layernorm_bwd(s["dy"], r, s["weight"], mean, rstd, dr=s["dr"])
        out.update(dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"])
        if s["residual"] is not None:
            out.update(residual=r, dresidual=g["dresidual"])
        return out
    if op == "conv":
        g = ss.ss_conv1d_bwd(s["dout"], s["x"], s["weight"], bias=s["bias"], window_in=s["window"], silu=c["silu"])
        out = dict(dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"])
        if s["window"] is not None:
            out["dwindow_in"] = g["dwindow_in"]
        return out
    if op == "xent":
        loss, lse = ss.ss_linear_xent(s["hidden"], s["weight"], s["targets"])
        out = dict(loss=loss, lse=lse)
        if c["grad"]:
            out.update(ss.ss_linear_xent_bwd(s["dloss"], s["hidden"], s["weight"], s["targets"], lse))
        return out
    if c["grad"]:
        loss, dlogits = ss.ss_distill_grad(s["dloss"], s["logits"], s["ids"], s["teacher"], temperature=c["temperature"])
        return dict(loss=loss, dlogits=dlogits)
    return dict(loss=ss.ss_distill(s["logits"], s["ids"], s["teacher"], temperature=c["temperature"]))


# -------------------------------------------------------------------------- bytes and operations

def work(case):
    es = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["D"]
        rs = 2 if case["res"] == "bf16" else 4
        stream = 4 * rs if case["residual"] else 0            # residual in and out, its gradient in and out
        return dict(bytes=n * (4 * es + stream) + 8 * case["rows"] + 16 * case["D"], flops=20 * n)
    if op == "conv":
        n = case["batch"] * case["L"] * case["Dm"]
        window = 24 * case["batch"] * case["Dm"] if case["window"] else 0
        return dict(bytes=3 * n * es + 40 * case["Dm"] + window, flops=(34 if case["silu"] else 18) * n)
    if op == "xent":
        T, D, V, n = case["tokens"], case["D"], case["V"], _trained(case)
        out = es * D * (T + V) if case["grad"] else 0
        return dict(bytes=es * D * (n + V) + out + 16 * T, flops=2 * n * D * V * (3 if case["grad"] else 1))
    n, V = _trained(case), case["V"]
    out = es * V * case["rows"] if case["grad"] else 0
    return dict(bytes=n * V * es + out + case["rows"] * (8 * case["K"] + 16), flops=n * V * (8 if case["grad"] else 4))


# --------------------------------------------------------------------- the definitions in 64 bits

def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def exact(case, seed):
    """The outputs by automatic differentiation of the definitions in doubles."""
    F = torch.nn.functional
    s = prepare(case, seed)
    op = case["op"]
    with torch.enable_grad():
        if op == "norm":
            x, w, b, dy = _leaf(s["x"]), _leaf(s["weight"]), _leaf(s["bias"]), s["dy"].double()
            res = None if s["residual"] is None else s["residual"].double()
            r = x if res is None else x + res
            y = F.layer_norm(r, r.shape[1:], w, b, EPS)
            loss = (y * dy).sum()
            if s["dr"] is not None:
                loss = loss + (r * s["dr"].double()).sum()
            dx, dw, db = torch.autograd.grad(loss, (x, w, b))
            var, mean = torch.var_mean(r.detach(), 1, correction=0)
            out = dict(y=y.detach(), mean=mean, rstd=1.0 / torch.sqrt(var + EPS), dx=dx, dweight=dw, dbias=db)
            if res is not None:
                out.update(residual=r.detach(), dresidual=dx)
            return out
        if op == "conv":
            x, w, b = _leaf(s["x"]), _leaf(s["weight"]), _leaf(s["bias"])
            win = _leaf(s["window"] if s["window"] is not None else torch.zeros(x.shape[0], x.shape[2], 3, device="cuda"))
            v = F.conv1d(torch.cat([win, x.transpose(1, 2)], 2), w[:, None, :], b, groups=w.shape[0])
            v = F.silu(v) if case["silu"] else v
            dx, dw, db, dwin = torch.autograd.grad(v, (x, w, b, win), s["dout"].double().transpose(1, 2))
            out = dict(dx=dx, dweight=dw, dbias=db)
            if s["window"] is not None:
                out["dwindow_in"] = dwin
            return out
        if op == "xent":
            T, D, V = case["tokens"], case["D"], case["V"]
            if T * D * V * (6 if case["grad"] else 2) > 12e12:
                return None
            h, w, t = _leaf(s["hidden"]), _leaf(s["weight"]), s["targets"].long()
            l = h @ w.t()
            loss = F.cross_entropy(l, t, ignore_index=-1, reduction="none")
            out = dict(loss=loss.detach(), lse=torch.logsumexp(l.detach(), 1) * (t >= 0))
            if case["grad"]:
                dh, dw = torch.autograd.grad(loss, (h, w), s["dloss"].double())
                out.update(dhidden=dh, dweight=dw)
            return out
        T = case["temperature"]
        parts, step = [], max(1, (1 << 28) // case["V"])
        for i in range(0, case["rows"], step):
            z = _leaf(s["logits"][i:i + step])
            ids = s["ids"][i:i + step].long()
            t = s["teacher"][i:i + step].double().masked_fill(ids < 0, -math.inf)
            lp = torch.log_softmax(t / T, 1)                   # (NaN in a row without entries)
            lq = torch.gather(torch.log_softmax(z / T, 1), 1, ids.clamp(min=0))
            some = ids >= 0
            loss = torch.where(some, torch.where(some, lp.exp() * lp, 0.0) - torch.where(some, lp.exp(), 0.0) * lq, 0.0).sum(1)
            part = [loss.detach()]
            if case["grad"]:
                part.append(torch.autograd.grad(loss, z, s["dloss"][i:i + step].double())[0])
            parts.append(part)
        return dict(zip(("loss", "dlogits"), (torch.cat(p) for p in zip(*parts))))
