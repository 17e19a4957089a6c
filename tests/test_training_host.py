"""Host-side checks of the training calls that need no GPU: bad arguments are refused before anything touches
a device; and the tests' own 64-bit gradients agree with differences of the definitions they belong to."""
import ctypes

import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import training_ref as ref

FAKE = 0x100000   # never dereferenced: these calls fail validation before any device access


def _no_gpu():
    torch = pytest.importorskip("torch")
    return not torch.cuda.is_available()


def test_layernorm_refuses_on_host():
    def call(x=FAKE, y=FAKE, w=FAKE, b=None, res=None, out=None, mean=None, rows=2, D=8, eps=1e-5, s=None):
        return ss.lib().ss_add_layernorm(x, res, w, b, out, y, mean, None, rows, D, eps, s, None)
    assert call(rows=-1) == 1 and call(D=-1) == 1 and call(D=1 << 20) == 2 and call(rows=1 << 40) == 2
    assert call(rows=0) == 0 and call(D=0) == 0
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None) == 1 and call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(x=FAKE + 1) == 3 and call(b=FAKE + 2) == 3 and call(mean=FAKE + 2) == 3 and call(out=FAKE + 3) == 3
    assert call(s=ctypes.byref(ss.NormStrides(ss.SS_F32, 9, 8, 8, 8, 8))) == 1
    assert call(s=ctypes.byref(ss.NormStrides(ss.SS_F32, ss.SS_F32, 8, 8, 8, 7))) == 1       # rows of y run into each other
    assert call(s=ctypes.byref(ss.NormStrides(ss.SS_F32, ss.SS_F32, -8, 8, 8, 8))) == 1
    if _no_gpu():
        assert call() == 4                                     # past the checks, stopped at the device


def test_layernorm_bwd_refuses_on_host():
    size = ss.lib().ss_add_layernorm_bwd_workspace_size

    def call(dy=FAKE, dr=None, r=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dres=None, dw=FAKE, db=FAKE, rows=2, D=8, s=None,
             ws=FAKE, nws=1 << 30):
        return ss.lib().ss_add_layernorm_bwd(dy, dr, r, w, mean, rstd, dx, dres, dw, db, rows, D, s, ws, nws, None)
    assert call(rows=-1) == 1 and call(D=-1) == 1 and call(D=1 << 20) == 2 and call(D=0) == 0
    for k in ("dy", "r", "w", "mean", "rstd", "dw", "db", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("dy", "r", "w", "mean", "rstd", "dx", "dw", "db"):
        assert call(**{k: FAKE + 1}) == 3, k
    assert call(ws=FAKE + 64) == 3 and call(nws=size(2, 8) - 1) == 1
    assert call(s=ctypes.byref(ss.NormGradStrides(ss.SS_F32, 2, 8, 8, 8, 8, 8))) == 1
    assert call(s=ctypes.byref(ss.NormGradStrides(ss.SS_F32, ss.SS_F32, 8, 8, 8, 7, 8))) == 1
    assert size(0, 8) == 0 and size(4, 0) == 0 and size(4, 1 << 20) == 0 and size(4, 8) > 0
    if _no_gpu():
        assert call() == 4 and call(rows=0) == 4


def test_conv1d_bwd_refuses_on_host():
    size = ss.lib().ss_conv1d_bwd_workspace_size

    def call(dout=FAKE, x=FAKE, w=FAKE, b=None, win=None, dwo=None, dx=FAKE, dw=FAKE, db=FAKE, dwi=None, batch=2, L=8, Dm=8, s=None,
             ws=FAKE, nws=1 << 30):
        return ss.lib().ss_conv1d_bwd(dout, x, w, b, win, dwo, dx, dw, db, dwi, batch, L, Dm, 1, s, ws, nws, None)
    assert call(batch=-1) == 1 and call(L=-1) == 1 and call(Dm=-1) == 1 and call(Dm=0) == 0
    assert call(batch=70000) == 2 and call(L=1 << 40) == 2
    for k in ("dout", "x", "w", "dx", "dw", "db", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("dout", "x", "w", "dx", "dw", "db"):
        assert call(**{k: FAKE + 1}) == 3, k
    assert call(win=FAKE + 2) == 3 and call(dwi=FAKE + 2) == 3 and call(ws=FAKE + 4) == 3
    assert call(nws=size(2, 8, 8) - 1) == 1
    assert call(s=ctypes.byref(ss.ConvGradStrides(7, 64, 8, 64, 8, 64, 8))) == 1
    assert call(s=ctypes.byref(ss.ConvGradStrides(ss.SS_F32, 64, 8, 64, 8, 0, 8))) == 1          # rows of dx share words
    assert call(s=ctypes.byref(ss.ConvGradStrides(ss.SS_F32, 64, -8, 64, 8, 64, 8))) == 1
    assert size(0, 8, 8) == 0 and size(2, 0, 8) == 0 and size(2, 8, 8) > 0
    if _no_gpu():
        assert call() == 4 and call(L=0) == 4


def test_distill_refuses_on_host():
    def call(z=FAKE, ids=FAKE, t=FAKE, loss=FAKE, rows=2, V=10, K=3, tau=1.0, s=None):
        return ss.lib().ss_distill(z, ids, t, loss, rows, V, K, tau, s, None)

    def grad(g=FAKE, z=FAKE, d=FAKE, rows=2, V=10, K=3, tau=1.0, s=None):
        return ss.lib().ss_distill_grad(g, z, FAKE, FAKE, FAKE, d, rows, V, K, tau, s, None)
    for f in (call, grad):
        assert f(rows=-1) == 1 and f(V=0) == 1 and f(K=-1) == 1 and f(V=1 << 30) == 2 and f(K=1025) == 2 and f(rows=1 << 40) == 2
        assert f(tau=0.0) == 1 and f(tau=-1.0) == 1 and f(tau=float("nan")) == 1 and f(tau=float("inf")) == 1
        assert f(rows=0) == 0 and f(z=None) == 1 and f(z=FAKE + 2) == 3
        assert f(s=ctypes.byref(ss.DistillStrides(3, 0, 10, 3, 3, 10, 1))) == 1
        assert f(s=ctypes.byref(ss.DistillStrides(0, 3, 10, 3, 3, 10, 1))) == 1
        assert f(s=ctypes.byref(ss.DistillStrides(0, 0, -1, 3, 3, 10, 1))) == 1
    assert call(ids=None) == 1 and call(t=None) == 1 and call(loss=None) == 1 and call(ids=FAKE + 1) == 3
    assert grad(g=None) == 1 and grad(d=None) == 1 and grad(g=FAKE + 2) == 3 and grad(d=FAKE + 1) == 3
    assert grad(s=ctypes.byref(ss.DistillStrides(0, 0, 10, 3, 3, 9, 1))) == 1                    # rows of dlogits run into each other
    assert grad(s=ctypes.byref(ss.DistillStrides(0, 0, 10, 3, 3, 10, -1))) == 1
    if _no_gpu():
        assert call() == 4 and call(K=0, ids=None, t=None) == 4 and grad() == 4


@pytest.mark.parametrize("tau,status", [(1e-31, 1), (1e-39, 1), (1e31, 1), (1e-30, 4), (1e30, 4)])
def test_distill_refuses_temperatures_without_a_normal_inverse(tau, status):
    if status == 4 and not _no_gpu():
        pytest.skip("the pointers are no memory")
    assert ss.lib().ss_distill(FAKE, FAKE, FAKE, FAKE, 2, 10, 3, tau, None, None) == status
    assert ss.lib().ss_distill_grad(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 10, 3, tau, None, None) == status


def test_linear_xent_refuses_on_host():
    size = ss.lib().ss_linear_xent_workspace_size

    def fwd(h=FAKE, w=FAKE, t=FAKE, loss=FAKE, lse=FAKE, T=4, V=10, D=8, s=None, ws=FAKE, nws=1 << 40):
        return ss.lib().ss_linear_xent(h, w, t, loss, lse, T, V, D, s, ws, nws, None)

    def bwd(g=FAKE, h=FAKE, w=FAKE, t=FAKE, lse=FAKE, dh=FAKE, dw=FAKE, T=4, V=10, D=8, s=None, ws=FAKE, nws=1 << 40):
        return ss.lib().ss_linear_xent_bwd(g, h, w, t, lse, dh, dw, T, V, D, s, ws, nws, None)
    for f, back in ((fwd, 0), (bwd, 1)):
        assert f(T=-1) == 1 and f(V=0) == 1 and f(D=0) == 1 and f(V=-3) == 1
        assert f(T=1 << 30) == 2 and f(V=1 << 30) == 2 and f(D=1 << 20) == 2
        for k in ("h", "w", "t", "lse", "ws"):
            assert f(**{k: None}) == 1, k
        for k in ("h", "w", "t", "lse"):
            assert f(**{k: FAKE + 1}) == 3, k
        assert f(ws=FAKE + 128) == 3 and f(nws=1000) == 1 and f(nws=size(4, 10, 8, 0, back)) in (4, 1)
        assert f(s=ctypes.byref(ss.XentStrides(5, 8, 8, 8, 8, 1))) == 1
        assert f(s=ctypes.byref(ss.XentStrides(0, -8, 8, 8, 8, 1))) == 1
        assert f(s=ctypes.byref(ss.XentStrides(0, 8, 7, 8, 8, 1))) == 1                          # rows of weight run into each other
        if _no_gpu():
            assert f() == 4
    assert fwd(T=0) == 0 and fwd(loss=None) == 1
    for k in ("g", "dh", "dw"):
        assert bwd(**{k: None}) == 1 and bwd(**{k: FAKE + 1}) == 3, k
    assert bwd(s=ctypes.byref(ss.XentStrides(0, 8, 8, 7, 8, 1))) == 1 and bwd(s=ctypes.byref(ss.XentStrides(0, 8, 8, 8, 7, 1))) == 1
    assert bwd(s=ctypes.byref(ss.XentStrides(0, 8, 8, 8, 8, -1))) == 1
    assert size(0, 10, 8, 0, 0) == 0 and size(4, 0, 8, 0, 0) == 0 and size(4, 10, 8, 9, 0) == 0
    # the workspace does not grow with the vocabulary beyond a piece of it
    assert size(4096, 1 << 20, 2048, ss.SS_BF16, 1) < (1 << 30) < 4096 * (1 << 20) * 2


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 64), torch.ones(64)
    one = torch.ones(2)
    for f in (lambda: ss.ss_add_layernorm(x, w), lambda: ss.ss_add_layernorm(x, w, residual=x),
              lambda: ss.ss_add_layernorm_bwd(x, x, w, one, one), lambda: ss.ss_conv1d_bwd(x[None], x[None], torch.zeros(64, 4)),
              lambda: ss.ss_distill(x, torch.zeros(2, 1, dtype=torch.int32), x[:, :1]),
              lambda: ss.ss_distill_grad(one, x, torch.zeros(2, 1, dtype=torch.int32), x[:, :1]),
              lambda: ss.ss_linear_xent(x, x, torch.zeros(2, dtype=torch.int32)),
              lambda: ss.ss_linear_xent_bwd(one, x, x, torch.zeros(2, dtype=torch.int32), one)):
        with pytest.raises(ValueError):
            f()


def _differences(f, x, g, h=1e-5):
    """Σ g · ∂f/∂x by central differences (f returns an array, g weights it)."""
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = (f() * g).sum()
        x[i] = keep - h
        d[i] = (up - (f() * g).sum()) / (2 * h)
        x[i] = keep
    return d


RNG = np.random.default_rng(5)


def _close(a, b):
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-8 * (1 + np.abs(b).max()))


def test_reference_of_the_norms_gradients():
    x, w, b, dy = RNG.standard_normal((3, 7)), RNG.standard_normal(7), RNG.standard_normal(7), RNG.standard_normal((3, 7))
    _, r, mean, rstd = ref.layernorm(x, None, w, b, 1e-2)
    d, dw, db = ref.layernorm_bwd(dy, r, w, mean, rstd)
    f = lambda: ref.layernorm(x, None, w, b, 1e-2)[0]                    # noqa: E731
    _close(d, _differences(f, x, dy))
    _close(dw, _differences(f, w, dy))
    _close(db, _differences(f, b, dy))


@pytest.mark.parametrize("L", [1, 2, 3, 6])
@pytest.mark.parametrize("silu", [True, False])
def test_reference_of_the_convolutions_gradients(L, silu):
    x, w, b = RNG.standard_normal((2, L, 3)), RNG.standard_normal((3, 4)), RNG.standard_normal(3)
    win, dout, dwo = RNG.standard_normal((2, 3, 3)), RNG.standard_normal((2, L, 3)), RNG.standard_normal((2, 3, 3))
    dx, dw, db, dwin = ref.conv1d_bwd(dout, x, w, b, win, dwo, silu)
    f = lambda: np.concatenate([a.ravel() for a in ref.conv1d(x, w, b, win, silu)])      # noqa: E731
    g = np.concatenate([dout.ravel(), dwo.ravel()])
    for got, arr in ((dx, x), (dw, w), (db, b), (dwin, win)):
        _close(got, _differences(f, arr, g))


def test_reference_of_the_cross_entropys_gradients():
    h, w, t, g = RNG.standard_normal((4, 3)), RNG.standard_normal((6, 3)), np.array([5, -1, 0, 5]), RNG.standard_normal(4)
    dh, dw = ref.xent_bwd(g, h, w, t)
    f = lambda: ref.xent(h, w, t)[0]                                     # noqa: E731
    _close(dh, _differences(f, h, g))
    _close(dw, _differences(f, w, g))


def test_reference_of_distillations_gradients():
    z, tau, g = RNG.standard_normal((4, 6)), 1.7, RNG.standard_normal(4)
    ids = np.array([[0, 5, 2], [1, -1, 1], [-1, -1, -1], [4, 4, 3]])
    t = RNG.standard_normal((4, 3))
    t[3, 2] = -np.inf
    loss, dz = ref.distill(z, ids, t, tau, g)
    assert loss[2] == 0 and not dz[2].any()
    _close(dz, _differences(lambda: ref.distill(z, ids, t, tau)[0], z, g))
