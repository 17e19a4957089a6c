"""The cross entropy where offsets into its tensors and its workspace pass 32 bits: many tokens, a large vocabulary, rows far apart."""
import ctypes

import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from xent_bounds import gradients, worst  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STRIDE = 4096


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    assert ss.device_error(clear=True) == 0


def apart(rows, D, dt):
    """[rows, D] of zeros, STRIDE elements from row to row."""
    return torch.zeros(rows, STRIDE, dtype=dt, device="cuda")[:, :D]


def backward(dloss, h, w, t, lse, dh, dw):
    """Through the C ABI, into outputs with strides of their own."""
    (T, D), V = h.shape, w.shape[0]
    s = ss.XentStrides(ss.SS_BF16 if h.dtype is torch.bfloat16 else ss.SS_F32, h.stride(0), w.stride(0), dh.stride(0), dw.stride(0), 1)
    n = ss.lib().ss_linear_xent_workspace_size(T, V, D, s.io_dtype, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = ss.lib().ss_linear_xent_bwd(dloss.data_ptr(), h.data_ptr(), w.data_ptr(), t.data_ptr(), lse.data_ptr(), dh.data_ptr(), dw.data_ptr(), T, V, D,
                                     ctypes.byref(s), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0


@pytest.mark.parametrize("io,T,V", [("bf16", 600000, 4000), ("f32", 560000, 2000), ("bf16", 300, 600000), ("bf16", 100, 600000), ("f32", 300, 560000)])
def test_rows_far_apart(io, T, V):
    """hidden and dhidden (or weight and dweight) of 2^31 elements and more from end to end; with 600000 tokens dl's piece as well."""
    D, dt = 64, DT[io]
    g = torch.Generator("cuda").manual_seed(1)
    many, wide = T > 100000, V > 100000
    h = apart(T, D, dt) if many else torch.zeros(T, D, dtype=dt, device="cuda")
    w = apart(V, D, dt) if wide else torch.zeros(V, D, dtype=dt, device="cuda")
    h.copy_(torch.randn(T, D, generator=g, device="cuda"))
    w.copy_(0.3 * torch.randn(V, D, generator=g, device="cuda"))
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[::9] = -1
    dloss = torch.randn(T, generator=g, device="cuda")
    loss, lse = ss.ss_linear_xent(h, w, t)
    dh = apart(T, D, dt) if many else torch.zeros_like(h)
    dw = apart(V, D, dt) if wide else torch.zeros_like(w)
    backward(dloss, h, w, t, lse, dh, dw)
    want = gradients(h.contiguous(), w.contiguous(), t, dloss)
    for k, v in (("dhidden", dh), ("dweight", dw)):
        assert worst({k: v}, want, k) <= 1.0, k


def test_partial_sums_of_many_tokens_over_a_large_vocabulary():
    """The forward pass leaves a maximum and a sum per token and half tile: 300000 x 8192 of them.  Some rows are compared."""
    T, V, D = 300000, 1 << 20, 8
    g = torch.Generator("cuda").manual_seed(2)
    h, w = torch.randn(T, D, generator=g, device="cuda").bfloat16(), torch.randn(V, D, generator=g, device="cuda").bfloat16()
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = ss.ss_linear_xent(h, w, t)
    at = torch.cat([torch.arange(0, T, 4999, device="cuda"), torch.arange(T - 40, T, device="cuda")])
    l = h[at].double() @ w.double().t()
    want = torch.logsumexp(l, 1)
    # logits' sums and the exponentials: see xent_bounds
    off = 4 * (D / 16 + 16) * 2.0 ** -23 * h[at].double().norm(dim=1) * w.double().norm(dim=1).max() + 2.0 ** -20
    assert bool(((lse[at].double() - want).abs() <= off).all())
    assert bool(((loss[at].double() - (want - l.gather(1, t[at].long()[:, None])[:, 0])).abs() <= off).all())
