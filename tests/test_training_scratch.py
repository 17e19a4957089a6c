"""Workspaces of the training calls through the C ABI: their contents before a call do not matter, nothing behind their
stated size is written, and neither is anything that the outputs held."""
import ctypes

import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 4096


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def stream():
    return torch.cuda.current_stream().cuda_stream


def with_scratch(nbytes, fill, call):
    """call(pointer of a workspace of nbytes filled with `fill`): checks what lies behind it."""
    ws = torch.full((nbytes + GUARD,), fill, dtype=torch.uint8, device="cuda")
    assert call(ws.data_ptr()) == 0
    torch.cuda.synchronize()
    assert bool((ws[nbytes:] == fill).all())


def nan_like(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(60, 3000, 200), (60, 3001, 203), (200, 3000, 200), (500, 3000, 200), (700, 2900, 131), (500, 700, 64)])
def test_cross_entropy(io, T, V, D):
    g = torch.Generator("cuda").manual_seed(T + V)
    h, w = torch.randn(T, D, generator=g, device="cuda").to(DT[io]), (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).to(DT[io])
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[torch.rand(T, generator=g, device="cuda") < 0.3] = -1
    L = ss.lib()
    for dloss in (torch.randn(T, generator=g, device="cuda"), torch.full((T,), 0.1, device="cuda")):
        got = []
        for fill in (0, 255, 0x7e):
            s = ss.XentStrides(ss.SS_BF16 if io == "bf16" else ss.SS_F32, D, D, D, D, 1)
            loss, lse, dh, dw = nan_like(T), nan_like(T), nan_like(T, D, dtype=DT[io]), nan_like(V, D, dtype=DT[io])
            n = L.ss_linear_xent_workspace_size(T, V, D, s.io_dtype, 0)
            with_scratch(n, fill, lambda ws: L.ss_linear_xent(h.data_ptr(), w.data_ptr(), t.data_ptr(), loss.data_ptr(), lse.data_ptr(), T, V, D,
                                                              ctypes.byref(s), ws, n, stream()))
            m = L.ss_linear_xent_workspace_size(T, V, D, s.io_dtype, 1)
            with_scratch(m, fill, lambda ws: L.ss_linear_xent_bwd(dloss.data_ptr(), h.data_ptr(), w.data_ptr(), t.data_ptr(), lse.data_ptr(),
                                                                  dh.data_ptr(), dw.data_ptr(), T, V, D, ctypes.byref(s), ws, m, stream()))
            got.append((loss, lse, dh, dw))
        for a in got:
            assert all(bool(torch.isfinite(v).all()) for v in a)
        for a in got[1:]:
            assert all(torch.equal(x, y) for x, y in zip(a, got[0]))


@pytest.mark.parametrize("rows,D", [(1, 64), (70, 256), (500, 111), (3000, 768)])
def test_layer_norm(rows, D):
    g = torch.Generator("cuda").manual_seed(rows)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
    dy, r, w, mean, rstd = rn(rows, D), rn(rows, D), rn(D), rn(rows), rn(rows).abs()
    L, n = ss.lib(), ss.lib().ss_add_layernorm_bwd_workspace_size(rows, D)
    got = []
    for fill in (0, 255):
        dx, dw, db = nan_like(rows, D), nan_like(D), nan_like(D)
        with_scratch(n, fill, lambda ws: L.ss_add_layernorm_bwd(dy.data_ptr(), None, r.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                                                dx.data_ptr(), None, dw.data_ptr(), db.data_ptr(), rows, D, None, ws, n, stream()))
        got.append((dx, dw, db))
    assert all(bool(torch.isfinite(a).all()) and torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("batch,L,Dm", [(1, 1, 32), (3, 50, 64), (2, 700, 33), (2, 5000, 256)])
def test_convolution(batch, L, Dm):
    g = torch.Generator("cuda").manual_seed(L)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
    dout, x, w = rn(batch, L, Dm), rn(batch, L, Dm), rn(Dm, 4)
    lib, n = ss.lib(), ss.lib().ss_conv1d_bwd_workspace_size(batch, L, Dm)
    got = []
    for fill in (0, 255):
        dx, dw, db, dwin = nan_like(batch, L, Dm), nan_like(Dm, 4), nan_like(Dm), nan_like(batch, Dm, 3)
        with_scratch(n, fill, lambda ws: lib.ss_conv1d_bwd(dout.data_ptr(), x.data_ptr(), w.data_ptr(), None, None, None, dx.data_ptr(), dw.data_ptr(),
                                                           db.data_ptr(), dwin.data_ptr(), batch, L, Dm, 1, None, ws, n, stream()))
        got.append((dx, dw, db, dwin))
    assert all(bool(torch.isfinite(a).all()) and torch.equal(a, b) for a, b in zip(*got))
