"""The training calls on operands that begin anywhere: a base in the middle of a 16-byte word, outputs given by the caller,
a first call that is captured.  Results are those of aligned copies: bit for bit where the same kernel takes both, else
within the calls' own tolerances."""
import subprocess
import sys
import os

import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def off(t):
    """A copy of t one element behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
    v = flat[1:1 + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def rn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def near(a, b, tol):
    a, b = a.double(), b.double()
    assert float((a - b).norm()) <= tol * float(b.norm()) + 1e-30


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned_bases(io):
    dt, tol = DT[io], (2e-6 if io == "f32" else 5e-3)
    x, dy, w, b, res = rn(1, 33, 256).to(dt), rn(2, 33, 256).to(dt), 1 + rn(3, 256), rn(4, 256), rn(5, 33, 256)
    a = ss.ss_add_layernorm(x, w, bias=b, residual=res)
    o = ss.ss_add_layernorm(off(x), off(w), bias=off(b), residual=off(res))
    for p, q in zip(o, a):
        near(p, q, tol)
    ga, go = ss.ss_add_layernorm_bwd(dy, a[1], w, a[2], a[3]), ss.ss_add_layernorm_bwd(off(dy), off(a[1]), off(w), off(a[2]), off(a[3]))
    for k in ga:
        near(go[k], ga[k], tol)
    c, dc, cw, win = rn(6, 2, 50, 64).to(dt), rn(7, 2, 50, 64).to(dt), rn(8, 64, 4), rn(9, 2, 64, 3)
    ga, go = ss.ss_conv1d_bwd(dc, c, cw, window_in=win), ss.ss_conv1d_bwd(off(dc), off(c), off(cw), window_in=off(win), dx=off(c))
    for k in ga:
        near(go[k], ga[k], tol)
    z, ids, t, g = rn(10, 6, 4096).to(dt), torch.arange(30, dtype=torch.int32, device="cuda").view(6, 5), rn(11, 6, 5), rn(12, 6)
    for p, q in zip(ss.ss_distill_grad(off(g), off(z), off(ids), off(t), dlogits=off(z)), ss.ss_distill_grad(g, z, ids, t)):
        near(p, q, tol)
    for T in (40, 400):
        h, head, tg, gl = rn(13, T, 64).to(dt), rn(14, 600, 64).to(dt), torch.arange(T, dtype=torch.int32, device="cuda"), rn(15, T)
        la, lo = ss.ss_linear_xent(h, head, tg), ss.ss_linear_xent(off(h), off(head), off(tg))
        assert torch.equal(la[0], lo[0]) and torch.equal(la[1], lo[1])
        ga, go = ss.ss_linear_xent_bwd(gl, h, head, tg, la[1]), ss.ss_linear_xent_bwd(off(gl), off(h), off(head), off(tg), off(la[1]))
        assert torch.equal(ga["dhidden"], go["dhidden"]) and torch.equal(ga["dweight"], go["dweight"])


def test_outputs_of_the_callers():
    x, w, res = rn(1, 20, 192).bfloat16(), 1 + rn(2, 192), rn(3, 20, 192)
    want = ss.ss_add_layernorm(x, w, residual=res)
    wide, rwide = torch.full((20, 200), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((20, 200), 7.0, device="cuda")
    y, r, mean, rstd = ss.ss_add_layernorm(x, w, residual=res, y=wide[:, 5:197], residual_out=rwide[:, :192])
    assert torch.equal(y, want[0]) and torch.equal(r, want[1]) and (wide[:, :5] == 7).all() and (wide[:, 197:] == 7).all() and (rwide[:, 192:] == 7).all()
    copy = torch.empty_like(x)
    y, r, mean, rstd = ss.ss_add_layernorm(x, w, residual_out=copy)      # without a residual: r is a copy of x
    assert r is copy and torch.equal(copy, x) and torch.equal(y, ss.ss_add_layernorm(x, w)[0])
    with pytest.raises(ValueError):
        ss.ss_add_layernorm(x, w, residual=res, y=wide)
    with pytest.raises(ValueError):
        ss.ss_distill_grad(rn(4, 3), rn(5, 3, 9), torch.zeros(3, 1, dtype=torch.int32, device="cuda"), rn(6, 3, 1), dlogits=rn(7, 3, 10))


def test_without_epsilon_and_without_gradients():
    x, w = rn(1, 5, 64), torch.ones(64, device="cuda")
    y, r, mean, rstd = ss.ss_add_layernorm(x, w, eps=0.0)
    near(y, torch.nn.functional.layer_norm(x.double(), (64,), eps=0.0), 2e-6)
    g = ss.ss_add_layernorm_bwd(torch.zeros_like(x), r, w, mean, rstd)
    assert not g["dx"].any() and not g["dweight"].any() and not g["dbias"].any()
    h, head, t = rn(2, 300, 64), rn(3, 100, 64), torch.zeros(300, dtype=torch.int32, device="cuda")
    loss, lse = ss.ss_linear_xent(h, head, t)
    for io in ("f32", "bf16"):
        d = ss.ss_linear_xent_bwd(torch.zeros(300, device="cuda"), h.to(DT[io]), head.to(DT[io]), t, lse)
        assert not d["dhidden"].any() and not d["dweight"].any()


def test_first_call_in_a_capture():
    """In a process of its own: nothing of the library has run on the device before the capture."""
    code = """
import torch, selective_state_space_scan_gb300 as ss
h = torch.randn(300, 64, device="cuda").bfloat16(); w = torch.randn(500, 64, device="cuda").bfloat16()
t = torch.arange(300, dtype=torch.int32, device="cuda"); g = torch.ones(300, device="cuda")
ss.lib(); torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    loss, lse = ss.ss_linear_xent(h, w, t)
    d = ss.ss_linear_xent_bwd(g, h, w, t, lse)
graph.replay(); torch.cuda.synchronize()
want = ss.ss_linear_xent(h, w, t); e = ss.ss_linear_xent_bwd(g, h, w, t, want[1])
torch.cuda.synchronize()
assert torch.equal(loss, want[0]) and torch.equal(d["dweight"], e["dweight"]) and torch.equal(d["dhidden"], e["dhidden"])
assert ss.device_error() == 0
print("same")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "same" in out.stdout, out.stderr[-2000:]
