"""Serving a stack of multi-head state space layers with random weights: packed prompts, then one
token of every request at a time, on one pool of cached states.

Every layer is residual norm (8 bits out) -> projection -> scan with its convolution -> projection;
the last norm's rows give the logits that ss_sample draws the next tokens from.  The projections
are plain matrix products; the codes of the 8-bit norm are exact in bfloat16.

    python examples/serve_stack.py            # three prompts, 16 tokens each
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_scan_gb300 as ss  # noqa: E402


class Layer:
    def __init__(self, g, width, H, P, G, N, slots, block=128):
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
        self.H, self.P, self.G, self.N, self.block = H, P, G, N, block
        self.C = H * P + 2 * G * N
        self.norm = torch.ones(width, device="cuda")
        self.w_in = (rn(H * P + self.C + H, width) / width ** 0.5).to(torch.bfloat16)
        self.w_out = (rn(width, H * P) / (H * P) ** 0.5).to(torch.bfloat16)
        self.conv_w, self.conv_b = 0.5 * rn(self.C, 4), 0.1 * rn(self.C)
        self.dt_bias = -4.0 - torch.rand(H, generator=g, device="cuda")
        self.A_log = torch.log(1.0 + 15.0 * torch.rand(H, generator=g, device="cuda"))
        self.D = torch.ones(H, device="cuda")
        self.state = torch.zeros(slots, H, P, N, device="cuda")
        self.window = torch.zeros(slots, self.C, 3, device="cuda")

    def __call__(self, x, residual, slots, cu_seqlens=None, fresh=None):
        """x [rows, width] bf16, residual [rows, width] fp32 (updated in place).  With cu_seqlens the rows are
        packed prompts, without it one token of every request."""
        y8, _, scale = ss.ss_add_rmsnorm_f8(x, self.norm, residual=residual, residual_out=residual, block=self.block)
        x8 = y8.to(torch.bfloat16) * scale.repeat_interleave(self.block, 1)[:, :x.shape[1]].to(torch.bfloat16)
        p = x8 @ self.w_in.t()
        HP = self.H * self.P
        z, xbc, dt = p[:, :HP], p[:, HP:HP + self.C], p[:, HP + self.C:]
        kw = dict(conv_b=self.conv_b, dt_bias=self.dt_bias, D=self.D, z=z, slots=slots)
        if cu_seqlens is None:
            y = ss.ss_heads_step(self.state, self.window, xbc, dt, self.conv_w, self.A_log, **kw)
        else:
            y = ss.ss_heads_fwd(xbc, dt, self.conv_w, self.A_log, self.state, self.window, cu_seqlens, fresh=fresh, **kw)
        return y @ self.w_out.t()


class Stack:
    def __init__(self, layers=2, width=768, H=24, P=64, G=1, N=128, vocab=1000, slots=8, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.slots = slots
        self.table = (torch.randn(vocab, width, generator=g, device="cuda")).to(torch.bfloat16)
        self.layers = [Layer(g, width, H, P, G, N, slots) for _ in range(layers)]
        self.norm = torch.ones(width, device="cuda")
        self.head = (torch.randn(vocab, width, generator=g, device="cuda") / width ** 0.5).to(torch.bfloat16)

    def __call__(self, tokens, slots, cu_seqlens=None, fresh=None):
        """Logits of every row of `tokens`."""
        x = self.table[tokens.long()]
        residual = torch.zeros(x.shape, device="cuda")
        for layer in self.layers:
            x = layer(x, residual, slots, cu_seqlens, fresh)
        y, _ = ss.ss_add_rmsnorm(x, self.norm, residual=residual, residual_out=residual)
        return y @ self.head.t()

    def generate(self, prompts, new_tokens, seed=0, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0):
        """prompts: lists of tokens, each on a slot of its own.  Returns [prompts, new_tokens] int32."""
        n, dev = len(prompts), "cuda"
        if not 0 < n <= self.slots or not all(prompts):
            raise ValueError(f"1 to {self.slots} prompts of a token or more are wanted")
        g = torch.Generator(dev).manual_seed(seed)
        lens = torch.tensor([0] + [len(p) for p in prompts])
        cu = torch.cumsum(lens, 0).to(torch.int32).to(dev)
        slots = torch.arange(n, dtype=torch.int32, device=dev)
        fresh = torch.ones(n, dtype=torch.int32, device=dev)
        packed = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=dev)
        logits = self(packed, slots, cu, fresh)[(cu[1:] - 1).long()]
        full = lambda v, t: torch.full((n,), v, dtype=t, device=dev)             # noqa: E731
        knobs = dict(temperature=full(temperature, torch.float32), top_k=full(top_k, torch.int32),
                     top_p=full(top_p, torch.float32), min_p=full(min_p, torch.float32))
        out = []
        for _ in range(new_tokens):
            noise = torch.empty(logits.shape, device=dev).exponential_(generator=g)
            out.append(ss.ss_sample(logits, noise, **knobs))
            logits = self(out[-1], slots)
        return torch.stack(out, 1)


def main():
    stack = Stack()
    prompts = [list(range(5, 305)), [7, 8, 9], list(range(100, 160))]
    tokens = stack.generate(prompts, 16)
    for p, t in zip(prompts, tokens.tolist()):
        print(f"{len(p)} tokens ->", *t)
    assert ss.device_error() == 0


if __name__ == "__main__":
    main()
