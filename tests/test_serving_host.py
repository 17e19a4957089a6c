"""Host-side checks of the serving calls that need no GPU: bad arguments are refused before anything
touches a device."""
import ctypes

import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import serving_ref as ref

FAKE = 0x10000   # never dereferenced: these calls fail validation before any device access


def _fwd(**kw):
    a = dict(xbc=FAKE, dt=FAKE, z=None, w=FAKE, b=None, tb=None, A=FAKE, D=None, y=FAKE, state=FAKE, window=FAKE, cu=FAKE,
             slots=None, fresh=None, n=2, T=9, H=4, P=64, G=2, N=128, pool=3, s=None, ws=FAKE, nws=1 << 30)
    a.update(kw)
    return ss.lib().ss_heads_fwd(a["xbc"], a["dt"], a["z"], a["w"], a["b"], a["tb"], a["A"], a["D"], a["y"], a["state"],
                                 a["window"], a["cu"], a["slots"], a["fresh"], a["n"], a["T"], a["H"], a["P"], a["G"], a["N"],
                                 a["pool"], a["s"], a["ws"], a["nws"], None)


def test_heads_fwd_refuses_on_host():
    assert _fwd(N=0) == 2 and _fwd(N=257) == 2 and _fwd(P=0) == 2 and _fwd(P=300) == 2
    assert _fwd(n=-1) == 1 and _fwd(T=-1) == 1 and _fwd(G=3) == 1 and _fwd(G=0) == 1 and _fwd(pool=-1) == 1
    assert _fwd(n=0) == 0 and _fwd(H=0, G=1) == 0
    assert _fwd(xbc=None) == 1 and _fwd(y=None) == 1 and _fwd(A=None) == 1 and _fwd(w=None) == 1 and _fwd(cu=None) == 1
    assert _fwd(state=None) == 1 and _fwd(window=None) == 1
    assert _fwd(pool=1) == 1                                   # slots by number, but too few of them
    assert _fwd(y=FAKE + 2) == 3 and _fwd(state=FAKE + 1) == 3 and _fwd(ws=FAKE + 64) == 3
    assert _fwd(ws=None) == 1 and _fwd(nws=1) == 1
    s = ss.HeadsStrides(5, 1000, 4, 0, 256)
    assert _fwd(s=ctypes.byref(s)) == 1                        # unknown type
    s = ss.HeadsStrides(ss.SS_BF16, 1000, 4, 0, 255)
    assert _fwd(s=ctypes.byref(s)) == 1                        # rows of y run into each other
    s = ss.HeadsStrides(ss.SS_BF16, -1, 4, 0, 256)
    assert _fwd(s=ctypes.byref(s)) == 1
    assert ss.lib().ss_heads_workspace_size(2, 9, 4, 64, 3, 128, ss.SS_F32) == 0
    assert ss.lib().ss_heads_workspace_size(2, 9, 4, 64, 2, 128, ss.SS_F32) > 0


def test_heads_step_refuses_on_host():
    def call(**kw):
        a = dict(n=2, H=4, P=64, G=2, N=128, pool=2, y=FAKE, state=FAKE, ws=FAKE)
        a.update(kw)
        return ss.lib().ss_heads_step(a["state"], FAKE, FAKE, FAKE, None, FAKE, None, None, FAKE, None, a["y"], None, a["n"],
                                      a["H"], a["P"], a["G"], a["N"], a["pool"], None, a["ws"], 1 << 20, None)
    assert call(N=300) == 2 and call(P=0) == 2
    assert call(n=-1) == 1 and call(G=3) == 1 and call(n=3) == 1 and call(state=None) == 1 and call(y=None) == 1
    assert call(ws=None) == 1 and call(n=0) == 0 and call(y=FAKE + 1) == 3


def test_norm_refuses_on_host():
    lib = ss.lib()

    def call(x=FAKE, y=FAKE, w=FAKE, rows=2, D=8, eps=1e-5, s=None):
        return lib.ss_add_rmsnorm(x, None, w, None, y, rows, D, eps, s, None)
    assert call(rows=-1) == 1 and call(D=-1) == 1 and call(D=1 << 20) == 2
    assert call(rows=0) == 0 and call(D=0) == 0
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None) == 1 and call(eps=-1.0) == 1
    assert call(eps=float("nan")) == 1 and call(x=FAKE + 1) == 3
    s = ss.NormStrides(ss.SS_F32, 9, 8, 8, 8, 8)
    assert call(s=ctypes.byref(s)) == 1
    s = ss.NormStrides(ss.SS_F32, ss.SS_F32, 8, 8, 8, 7)
    assert call(s=ctypes.byref(s)) == 1                        # rows of y run into each other
    f8 = lambda block, scale=FAKE: lib.ss_add_rmsnorm_f8(FAKE, None, FAKE, None, FAKE, scale, 2, 64, block, 1e-5, None, None)  # noqa: E731
    assert f8(48) == 2 and f8(-32) == 2 and f8(512) == 2 and f8(64, None) == 1


def test_sample_refuses_on_host():
    def call(l=FAKE, e=FAKE, out=FAKE, rows=1, V=10, io=0, lr=10, er=10, k=None):
        return ss.lib().ss_sample(l, e, None, k, None, None, out, rows, V, io, lr, er, None)
    assert call(rows=-1) == 1 and call(V=0) == 1 and call(V=(1 << 20) + 1) == 2 and call(io=7) == 1
    assert call(rows=0) == 0
    assert call(l=None) == 1 and call(e=None) == 1 and call(out=None) == 1 and call(lr=-1) == 1
    assert call(l=FAKE + 2) == 3 and call(l=FAKE + 1, io=1) == 3 and call(k=FAKE + 2) == 3


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        ss.ss_add_rmsnorm(x, torch.ones(64))
    with pytest.raises(ValueError):
        ss.ss_sample(x, x)
    with pytest.raises(ValueError):
        ss.ss_heads_step(torch.zeros(2, 1, 32, 16), torch.zeros(2, 64, 3), x, torch.zeros(2, 1), torch.zeros(64, 4), torch.zeros(1))
    with pytest.raises(ValueError):                            # channels that no G explains
        ss.ss_heads_step(torch.zeros(2, 1, 32, 16), torch.zeros(2, 70, 3), torch.zeros(2, 70), torch.zeros(2, 1),
                         torch.zeros(70, 4), torch.zeros(1))


def test_reference_of_the_scan_has_a_closed_form():
    """Constant inputs: S settles at dt*x*B / (1 - a), the geometric series; pins the test's own reference."""
    H, P, N, L = 1, 2, 3, 4000
    C = H * P + 2 * N
    w = np.zeros((C, 4))
    w[:, 3] = 1.0
    xbc = np.tile(np.linspace(0.5, 1.5, C), (L, 1))
    y, S, W = ref.heads(xbc, np.zeros((L, 1)), w, None, None, np.zeros(1), None, None, np.zeros((H, P, N)), np.zeros((C, 3)), P, N)
    u = ref.silu(xbc[0])
    dt = np.log(2.0)
    limit = dt * np.outer(u[:P], u[P:P + N]) / (1 - np.exp(-dt))
    np.testing.assert_allclose(S[0], limit, rtol=1e-12)
    np.testing.assert_allclose(y[-1], limit @ u[P + N:], rtol=1e-12)
    np.testing.assert_array_equal(W, xbc[-3:].T)


def test_reference_of_the_codes():
    """Every e4m3 value is its own nearest, and the middle between two goes to the even one."""
    v = [m / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8, 16)][:-1] + [k * 2.0 ** -9 for k in range(8)]
    v = np.unique(np.array(v))
    np.testing.assert_array_equal(ref.e4m3_nearest(v), v)
    mid = (v[:-1] + v[1:]) / 2
    even = np.where(np.round(v[:-1] / (v[1:] - v[:-1])) % 2 == 0, v[:-1], v[1:])
    np.testing.assert_array_equal(ref.e4m3_nearest(mid), even)


def test_reference_of_the_sampler():
    l = np.array([1.0, 3.0, 3.0, -np.inf, 2.0], np.float32)
    e = np.ones(5, np.float32)
    assert ref.sample_row(l, e) == 1 and ref.sample_row(l, e, temperature=0) == 1
    assert ref.sample_row(l, np.array([1e-9, 1, 0.5, 1, 1], np.float32), top_k=2) == 2
    assert ref.sample_row(l, np.array([1, 1, 1e-9, 1, 1], np.float32), top_k=1) == 1
    assert ref.sample_row(l, np.array([1e-9, 1, 1, 1, 1], np.float32), top_p=0.9) == 1
    assert ref.sample_row(l, np.array([1e-9, 1, 1, 1, 1], np.float32)) == 0
    assert ref.sample_row(np.full(3, -np.inf, np.float32), e[:3]) == -1
