"""Workloads of the operators that serve a stack of state space layers.

Four operators, each in a plain form (elementary torch operations in 32 bits) and as the library's
call, chosen by ``own``:

  heads_fwd    the multi-head selective scan with its short causal convolution, for packed prompts
               of different lengths, from and into a pool of cached states
  heads_step   the same for one token of every request
  norm         residual addition and root-mean-square norm, with outputs in 8 bits and their scales
               (or in the input's type)
  sample       temperature, top-k, top-p and min-p sampling from given random numbers

``listed()`` gives fixed cases, ``draw(rng)`` further ones of the same ranges, ``prepare`` what a
program holds before the call, ``run`` one call, ``work`` the bytes and operations it cannot do
without, ``exact`` the result in 64 bits.
"""
import math
import random

import torch

own = False

CHUNK = 128            # steps per chunk of the plain scan
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one short user turn appended to a running conversation: latency counts
        dict(name="turn of 45 tokens", op="heads_fwd", seqs=1, longest=45, H=24, P=64, G=1, N=128, io="bf16", even=True,
             gate=True, fresh=0.0),
        # a batch of prompts as they arrive, packed without padding; some continue from their slots
        dict(name="ragged prompts", op="heads_fwd", seqs=13, longest=2047, H=24, P=64, G=1, N=128, io="bf16", even=False,
             gate=True, fresh=0.5),
        # one long document on a narrow layer: few heads, so the time axis has to be split
        dict(name="document of 32k tokens", op="heads_fwd", seqs=1, longest=32768, H=24, P=64, G=1, N=128, io="bf16",
             even=True, gate=True, fresh=1.0),
        # a wide layer on full prompts: the largest call
        dict(name="wide layer prompts", op="heads_fwd", seqs=4, longest=8192, H=80, P=64, G=1, N=128, io="bf16", even=True,
             gate=True, fresh=1.0),
        # 32-bit activations, two groups of B and C, 64 states, the gate applied by the caller
        dict(name="float32 prompts", op="heads_fwd", seqs=8, longest=1024, H=24, P=64, G=2, N=64, io="f32", even=False,
             gate=False, fresh=1.0),
        # one request's next token: latency alone
        dict(name="one token", op="heads_step", batch=1, H=24, P=64, G=1, N=128, io="bf16", gate=True),
        # a serving batch, odd, on a 4096-channel layer
        dict(name="tokens of 61 requests", op="heads_step", batch=61, H=64, P=64, G=1, N=128, io="bf16", gate=True),
        # a large serving batch in 32-bit activations
        dict(name="tokens of 256 requests", op="heads_step", batch=256, H=80, P=64, G=8, N=64, io="f32", gate=True),
        # the norm before a layer while decoding: few rows
        dict(name="norm of 61 rows", op="norm", rows=61, D=2560, io="bf16", res="f32", out="f8", block=0),
        # the same over prompts, scales per 128 columns for a blockwise 8-bit projection
        dict(name="norm of 32k rows", op="norm", rows=32768, D=2560, io="bf16", res="f32", out="f8", block=128),
        # the next token of one conversation
        dict(name="sample one row", op="sample", rows=1, V=50257, io="f32"),
        # the next tokens of a batch on a large vocabulary, every row with its own settings
        dict(name="sample 192 rows", op="sample", rows=192, V=128000, io="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _not_3k(n):
    """Sizes of 3072 are left to the configurations that have them: none here."""
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(("heads_fwd", "heads_fwd", "heads_step", "norm", "sample"))
    io = rng.choice(("bf16", "bf16", "f32"))
    if op in ("heads_fwd", "heads_step"):
        P, N = rng.choice((32, 64, 64, 64, 128)), rng.choice((16, 64, 128, 128))
        G = rng.choice((1, 1, 2, 4))
        H = G * max(1, _log_int(rng, 8, 80) * 64 // (P * G))
        if H * P == 3072:
            H += G
        if op == "heads_step":
            return dict(op=op, batch=_log_int(rng, 1, 256), H=H, P=P, G=G, N=N, io=io, gate=rng.random() < 0.8)
        seqs = _log_int(rng, 1, 16)
        longest = _not_3k(_log_int(rng, 1, 32768 // seqs))
        return dict(op=op, seqs=seqs, longest=longest, H=H, P=P, G=G, N=N, io=io, even=rng.random() < 0.3,
                    gate=rng.random() < 0.8, fresh=rng.choice((0.0, 0.5, 1.0)))
    if op == "norm":
        D = _not_3k(_log_int(rng, 64, 8192))
        out = rng.choice(("f8", "f8", "io"))
        if rng.random() < 0.7:
            D = _not_3k(-(-D // 128) * 128)
        return dict(op=op, rows=_not_3k(_log_int(rng, 1, 32768)), D=D, io=io, res=rng.choice(("f32", "bf16")), out=out,
                    block=rng.choice((0, 64, 128)) if out == "f8" else 0)
    return dict(op=op, rows=_log_int(rng, 1, 192), V=_not_3k(_log_int(rng, 1000, 128000)), io=io)


# ----------------------------------------------------------------------------------- the inputs

def _io(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator("cuda").manual_seed(int(seed) % (1 << 62))


def _lengths(case):
    """Lengths of the packed sequences: all the longest, or one of them that long and the others spread
    below it, with an empty one where there are four or more.  They are part of the case: a shape."""
    n, top = case["seqs"], case["longest"]
    if case["even"] or n == 1:
        return [top] * n
    r = random.Random(1000003 * n + top)
    lens = [r.randint(1, top) for _ in range(n)]
    first, empty = r.sample(range(n), 2)
    lens[first] = top
    if n >= 4:
        lens[empty] = 0
    return lens


def _layer(case, g):
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    C = H * P + 2 * G * N
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g, device="cuda")           # noqa: E731
    return dict(conv_w=0.5 * rn(C, 4), conv_b=0.1 * rn(C), dt_bias=-ru(H), A_log=torch.log(1.0 + 15.0 * ru(H)),
                D=1.0 + 0.1 * rn(H))


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], dict(case=case)
    rn = lambda *sh: torch.randn(*sh, generator=g, device="cuda")         # noqa: E731
    if op == "norm":
        io, rows, D = _io(case), case["rows"], case["D"]
        s.update(x=rn(rows, D).to(io), residual=(3.0 * rn(rows, D)).to(torch.bfloat16 if case["res"] == "bf16" else torch.float32),
                 weight=1.0 + 0.2 * rn(D))
        return s
    if op == "sample":
        io, rows, V = _io(case), case["rows"], case["V"]
        ru = torch.rand(rows, 4, generator=g, device="cuda")
        # every fifth row greedy, temperatures 0.5 to 1.2; each filter off in some of the rows
        temp = torch.where(ru[:, 0] < 0.2, torch.zeros(()).cuda(), 0.5 + 0.7 * ru[:, 0])
        top_k = torch.where(ru[:, 1] < 0.3, torch.zeros((), dtype=torch.int64).cuda(), (1 + 200 * ru[:, 1]).long()).to(torch.int32)
        top_p = torch.where(ru[:, 2] < 0.3, torch.ones(()).cuda(), 0.6 + 0.39 * ru[:, 2])
        min_p = torch.where(ru[:, 3] < 0.5, torch.zeros(()).cuda(), 0.1 * ru[:, 3])
        noise = torch.empty(rows, V, device="cuda").exponential_(generator=g)
        s.update(logits=(2.5 * rn(rows, V)).to(io), noise=noise, temperature=temp, top_k=top_k, top_p=top_p, min_p=min_p)
        return s
    io, H, P, G, N = _io(case), case["H"], case["P"], case["G"], case["N"]
    C = H * P + 2 * G * N
    s.update(_layer(case, g))
    if op == "heads_fwd":
        lens = _lengths(case)
        n, T = len(lens), sum(lens)
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        s.update(lens=lens, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        s["fresh"] = (torch.rand(n, generator=g, device="cuda") < case["fresh"]).to(torch.int32)
    else:
        n = T = case["batch"]
    pool = n + 1
    s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32)
    s.update(state=0.5 * rn(pool, H, P, N), window=rn(pool, C, 3))
    # one projection gives z, xbc and the time steps side by side; the operators read its columns in place
    wide = torch.empty(T, H * P + C + H, dtype=io, device="cuda")
    step = max(1, (1 << 28) // wide.shape[1])
    for i in range(0, T, step):
        wide[i:i + step] = rn(min(step, T - i), wide.shape[1]).to(io)
    wide[:, H * P + C:] = (rn(T, H) - 4.0).to(io)
    s.update(z=wide[:, :H * P] if case["gate"] else None, xbc=wide[:, H * P:H * P + C], dt_raw=wide[:, H * P + C:])
    return s


# -------------------------------------------------------------------------------- the plain forms

def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _conv(e, w, b, L):
    """silu(b + sum_k w[:, k] e[t + k]) over the time axis, the last but one of e."""
    return _silu(b + w[:, 0] * e[:, 0:L] + w[:, 1] * e[:, 1:L + 1] + w[:, 2] * e[:, 2:L + 2] + w[:, 3] * e[:, 3:L + 3])


def _plain_fwd(s):
    c = s["case"]
    H, P, G, N = c["H"], c["P"], c["G"], c["N"]
    lens, cu, slots = s["lens"], s["cu_seqlens"].long(), s["slots"].long()
    n, T = len(lens), s["xbc"].shape[0]
    nc = max(1, -(-max(lens) // CHUNK))
    L = nc * CHUNK
    length = cu[1:] - cu[:-1]
    pos = torch.arange(L, device="cuda")
    valid = pos[None, :] < length[:, None]                                     # [n, L]
    at = torch.where(valid, cu[:-1, None] + pos[None, :], 0)
    keep = (s["fresh"] == 0).float()
    S0 = s["state"][slots] * keep[:, None, None, None]
    win = s["window"][slots] * keep[:, None, None]
    e = torch.cat([win.transpose(1, 2), s["xbc"].float()[at] * valid[..., None]], 1)   # [n, 3 + L, C]
    u = _conv(e, s["conv_w"], s["conv_b"], L)
    new_win = torch.gather(e, 1, (length[:, None] + torch.arange(3, device="cuda"))[..., None].expand(-1, -1, e.shape[2]))
    del e
    dt = _softplus(s["dt_raw"].float() + s["dt_bias"])[at] * valid[..., None]        # [n, L, H]
    x = u[..., :H * P].reshape(n, nc, CHUNK, H, P)
    B = u[..., H * P:H * P + G * N].reshape(n, nc, CHUNK, G, N).permute(0, 1, 3, 2, 4)
    C = u[..., H * P + G * N:].reshape(n, nc, CHUNK, G, N).permute(0, 1, 3, 2, 4)
    a = (dt * -torch.exp(s["A_log"])).reshape(n, nc, CHUNK, H).permute(0, 1, 3, 2)
    cs = torch.cumsum(a, -1)                                                   # [n, nc, H, CHUNK]
    dtc = dt.reshape(n, nc, CHUNK, H).permute(0, 1, 3, 2)
    xh = x.permute(0, 1, 3, 2, 4)                                              # [n, nc, H, CHUNK, P]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp(torch.where(tri, cs[..., :, None] - cs[..., None, :], -math.inf))
    score = torch.matmul(C, B.transpose(-1, -2))                               # [n, nc, G, CHUNK, CHUNK]
    M = decay.reshape(n, nc, G, H // G, CHUNK, CHUNK) * score[:, :, :, None]
    del decay
    M = M.reshape(n, nc, H, CHUNK, CHUNK) * dtc[..., None, :]
    y = torch.matmul(M, xh)                                                    # [n, nc, H, CHUNK, P]
    del M
    tail = torch.exp(cs[..., -1:] - cs) * dtc                                  # decay from a step to the chunk's end
    xt = (xh * tail[..., None]).transpose(-1, -2).reshape(n, nc, G, H // G, P, CHUNK)
    Z = torch.matmul(xt, B[:, :, :, None]).reshape(n, nc, H, P * N)
    tot = torch.cat([torch.zeros(n, 1, H, device="cuda"), torch.cumsum(cs[..., -1], 1)], 1)   # [n, nc + 1, H]
    tot = tot.transpose(1, 2)                                                  # log decay before chunk i
    # state before chunk i: sum over j < i of exp(tot_i - tot_{j+1}) Z_j, and exp(tot_i) S0
    low = torch.ones(nc + 1, nc, dtype=torch.bool, device="cuda").tril(-1)
    W = torch.exp(torch.where(low, tot[..., :, None] - tot[..., None, 1:], -math.inf))         # [n, H, nc + 1, nc]
    S = torch.matmul(W, Z.transpose(1, 2)).reshape(n, H, nc + 1, P, N)
    del Z, W
    S = S + torch.exp(tot)[..., None, None] * S0[:, :, None]
    Sin = S[:, :, :nc].permute(0, 2, 1, 4, 3).reshape(n, nc, G, H // G, N, P)
    off = torch.matmul(C[:, :, :, None], Sin).reshape(n, nc, H, CHUNK, P)
    y = y + off * torch.exp(cs)[..., None] + s["D"][:, None, None] * xh
    y = y.permute(0, 1, 3, 2, 4).reshape(n, L, H * P)[valid]                    # packed again, in order
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slots] = S[:, :, nc]
    s["window"][slots] = new_win.transpose(1, 2)
    return dict(y=y.to(s["xbc"].dtype), state=s["state"], window=s["window"])


def _plain_step(s):
    c = s["case"]
    H, P, G, N, n = c["H"], c["P"], c["G"], c["N"], c["batch"]
    slots = s["slots"].long()
    win = s["window"][slots]
    e = torch.cat([win, s["xbc"].float()[..., None]], -1)                       # [n, C, 4]
    u = _silu(s["conv_b"] + (e * s["conv_w"]).sum(-1))
    x = u[:, :H * P].reshape(n, H, P)
    B = u[:, H * P:H * P + G * N].reshape(n, G, 1, 1, N).expand(-1, -1, H // G, 1, -1).reshape(n, H, 1, N)
    C = u[:, H * P + G * N:].reshape(n, G, 1, 1, N).expand(-1, -1, H // G, 1, -1).reshape(n, H, 1, N)
    dt = _softplus(s["dt_raw"].float() + s["dt_bias"])
    a = torch.exp(dt * -torch.exp(s["A_log"]))
    S = s["state"][slots] * a[..., None, None] + (dt[..., None] * x)[..., None] * B
    y = ((S * C).sum(-1) + s["D"][:, None] * x).reshape(n, H * P)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slots] = S
    s["window"][slots] = e[..., 1:]
    return dict(y=y.to(s["xbc"].dtype), state=s["state"], window=s["window"])


EPS = 1e-5
F8_MAX = 448.0
AMAX_MIN = 1e-30


def _plain_norm(s):
    c = s["case"]
    r = s["x"].float() + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"]
    out = dict(residual=r.to(s["residual"].dtype))
    if c["out"] == "io":
        out["y"] = y.to(s["x"].dtype)
        return out
    rows, D = y.shape
    blk = c["block"] or D
    nb = -(-D // blk)
    yb = torch.nn.functional.pad(y, (0, nb * blk - D)).reshape(rows, nb, blk)
    scale = torch.clamp(yb.abs().amax(-1), min=AMAX_MIN) / F8_MAX
    out["y"] = (yb / scale[..., None]).to(F8).reshape(rows, nb * blk)[:, :D]
    out["scale"] = scale
    return out


def _plain_sample(s):
    l = s["logits"].float()
    l = torch.clamp(torch.where(torch.isnan(l), -math.inf, l), max=torch.finfo(torch.float32).max)
    V = l.shape[1]
    ls, idx = torch.sort(l, dim=-1, descending=True, stable=True)
    T = torch.where(s["temperature"] > 0, s["temperature"], 1.0)[:, None]
    w = torch.exp((ls - ls[:, :1]) / T)
    rank = torch.arange(V, device="cuda")[None, :]
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    wk = torch.where(rank < k, w, 0.0)
    cum = torch.cumsum(wk, -1)
    p = torch.where(s["top_p"] < 1, s["top_p"], math.inf)[:, None]
    keep = (rank < k) & (cum - wk < p * cum[:, -1:]) & (w >= s["min_p"][:, None])
    greedy = (s["temperature"] <= 0)[:, None]
    keep = torch.where(greedy, False, keep) | (rank == 0)
    key = torch.where(keep, w / torch.gather(s["noise"], 1, idx), -1.0)
    best = key.amax(-1, keepdim=True)
    token = torch.where(key == best, idx, V).amin(-1)
    return torch.where(ls[:, 0] == -math.inf, -1, token).to(torch.int32)


def run(s):
    op = s["case"]["op"]
    if not own:
        return dict(heads_fwd=_plain_fwd, heads_step=_plain_step, norm=_plain_norm, sample=_plain_sample)[op](s)
    import selective_state_space_scan_gb300 as ss
    if op == "heads_fwd":
        y = ss.ss_heads_fwd(s["xbc"], s["dt_raw"], s["conv_w"], s["A_log"], s["state"], s["window"], s["cu_seqlens"],
                            conv_b=s["conv_b"], dt_bias=s["dt_bias"], D=s["D"], z=s["z"], slots=s["slots"], fresh=s["fresh"])
        return dict(y=y, state=s["state"], window=s["window"])
    if op == "heads_step":
        y = ss.ss_heads_step(s["state"], s["window"], s["xbc"], s["dt_raw"], s["conv_w"], s["A_log"], conv_b=s["conv_b"],
                             dt_bias=s["dt_bias"], D=s["D"], z=s["z"], slots=s["slots"])
        return dict(y=y, state=s["state"], window=s["window"])
    if op == "norm":
        if s["case"]["out"] == "io":
            y, r = ss.ss_add_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return dict(y=y, residual=r)
        y, r, scale = ss.ss_add_rmsnorm_f8(s["x"], s["weight"], residual=s["residual"], eps=EPS, block=s["case"]["block"])
        return dict(y=y, residual=r, scale=scale)
    return ss.ss_sample(s["logits"], s["noise"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                        min_p=s["min_p"])


# -------------------------------------------------------------------------- bytes and operations

def work(case):
    es = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["D"]
        rs = 2 if case["res"] == "bf16" else 4
        nb = -(-case["D"] // (case["block"] or case["D"]))
        o = n * es if case["out"] == "io" else n + 4 * case["rows"] * nb
        return dict(bytes=n * (es + 2 * rs) + o + 4 * case["D"], flops=6 * n)
    if op == "sample":
        n = case["rows"] * case["V"]
        return dict(bytes=n * (es + 4) + 24 * case["rows"], flops=4 * n)
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    C = H * P + 2 * G * N
    T, n = (case["batch"],) * 2 if op == "heads_step" else (sum(_lengths(case)), case["seqs"])
    per_token = es * (C + H + H * P * (2 if case["gate"] else 1))
    cache = 4 * (H * P * N + 3 * C)
    reads = 1.0 if op == "heads_step" else 1.0 - case["fresh"]
    weights = 4 * (5 * C + 3 * H)
    # the recurrence itself: per head and token P*N multiply-adds of the update, as many for the output, and the decay
    return dict(bytes=T * per_token + n * cache * (1 + reads) + weights, flops=T * (5 * H * P * N + 12 * C))


# --------------------------------------------------------------------- the definitions in 64 bits

def _exact_tokens(s, x_rows, dt_rows, z_rows, state, window):
    """One step of every request whose row is given, in doubles: the definition itself."""
    c = s["case"]
    H, P, G, N = c["H"], c["P"], c["G"], c["N"]
    n = x_rows.shape[0]
    e = torch.cat([window, x_rows[..., None]], -1)
    v = (e * s["conv_w"].double()).sum(-1) + s["conv_b"].double()
    u = v * torch.sigmoid(v)
    x, B, C = u[:, :H * P].view(n, H, P), u[:, H * P:H * P + G * N].view(n, G, N), u[:, H * P + G * N:].view(n, G, N)
    dt = torch.logaddexp(dt_rows + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    a = torch.exp(-dt * torch.exp(s["A_log"].double()))
    B, C = B.repeat_interleave(H // G, 1), C.repeat_interleave(H // G, 1)
    state = state * a[..., None, None] + torch.einsum("nhp,nhk->nhpk", x * dt[..., None], B)
    y = torch.einsum("nhpk,nhk->nhp", state, C) + s["D"].double()[:, None] * x
    y = y.reshape(n, H * P)
    if z_rows is not None:
        y = y * z_rows * torch.sigmoid(z_rows)
    return y, state, e[..., 1:]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        r = s["x"].double() + s["residual"].double()
        y = r / torch.sqrt((r ** 2).sum(-1, keepdim=True) / r.shape[1] + EPS) * s["weight"].double()
        if case["out"] == "io":
            return dict(y=y, residual=r)
        blk = case["block"] or case["D"]
        parts = [y[:, i:i + blk] for i in range(0, case["D"], blk)]
        scales = [(p.abs().max(-1).values / F8_MAX) for p in parts]
        q = torch.cat([p / v[:, None] for p, v in zip(parts, scales)], 1)
        # e4m3: three bits after the point of a number in [1, 2), exponents down to -6
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(q.abs().clamp(min=1e-300))), min=-6.0) - 3.0)
        return dict(y=torch.round(q / step) * step, residual=r, scale=torch.stack(scales, 1))
    if op == "sample":
        return None                                           # whole numbers: held to the plain form's
    slots = s["slots"].long()
    state, window = s["state"].double(), s["window"].double()
    if op == "heads_step":
        y, S, W = _exact_tokens(s, s["xbc"].double(), s["dt_raw"].double(), None if s["z"] is None else s["z"].double(),
                                state[slots], window[slots])
        state[slots], window[slots] = S, W
        return dict(y=y, state=state, window=window)
    H, P, N = case["H"], case["P"], case["N"]
    elems = len(s["lens"]) * H * P * N
    if max(s["lens"], default=0) * (2.5e-4 + elems * 1.2e-10) > 18.0:
        return None
    keep = (s["fresh"] == 0).double()
    S, W = state[slots] * keep[:, None, None, None], window[slots] * keep[:, None, None]
    start = s["cu_seqlens"].long()[:-1]
    order = sorted(range(len(s["lens"])), key=lambda i: -s["lens"][i])           # the longest first
    ranked = torch.tensor(order, device="cuda")
    S, W, start = S[ranked], W[ranked], start[ranked]
    y = torch.empty(s["xbc"].shape[0], H * P, dtype=torch.float64, device="cuda")
    m = len(order)
    for t in range(max(s["lens"], default=0)):
        while m and s["lens"][order[m - 1]] <= t:
            m -= 1
        rows = start[:m] + t
        z = None if s["z"] is None else s["z"][rows].double()
        y[rows], S[:m], W[:m] = _exact_tokens(s, s["xbc"][rows].double(), s["dt_raw"][rows].double(), z, S[:m], W[:m])
    state[slots[ranked]], window[slots[ranked]] = S, W
    return dict(y=y, state=state, window=window)
