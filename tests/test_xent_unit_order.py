"""The cross entropy's two gradient products share one launch, and a pair of CTAs takes tiles of dweight and slices of
dhidden in turn.  Sizes where tiles of dweight come first and the same pair has dhidden's afterwards (a slice of the
vocabulary no longer than the tokens), short slices among them: every element against the definition in 64 bits, and the same bits every time."""
import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from xent_bounds import gradients, worst  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(1524, 13459, 128), (16384, 12800, 64), (3000, 2000, 2560), (8192, 5000, 1000)])
def test_dhidden_behind_dweight(io, T, V, D):
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(T)
    h = torch.randn(T, D, generator=g, device="cuda").to(dt)
    w = (1.5 / D ** 0.5 * torch.randn(V, D, generator=g, device="cuda")).to(dt)
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[::11] = -1
    dloss = torch.randn(T, generator=g, device="cuda")
    loss, lse = ss.ss_linear_xent(h, w, t)
    first = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)
    want = gradients(h, w, t, dloss)
    for k in ("dhidden", "dweight"):
        assert worst(first, want, k) <= 1.0, k
    for _ in range(10):
        again = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)
        assert torch.equal(again["dhidden"], first["dhidden"]) and torch.equal(again["dweight"], first["dweight"])
