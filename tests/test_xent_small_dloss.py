"""Tokens whose dloss is a small part of the largest: their rows of dhidden, element by element and so each by itself, are as
exact as the others' (a norm over the whole tensor would not see them)."""
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
@pytest.mark.parametrize("T", [40, 200, 450])
@pytest.mark.parametrize("most", [1.0, 2.0 ** 40, 2.0 ** -60])
def test_every_row(io, T, most):
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    V, D = 20000, 128
    g = torch.Generator("cuda").manual_seed(T)
    h = torch.randn(T, D, generator=g, device="cuda").to(dt)
    w = (1.5 / D ** 0.5 * torch.randn(V, D, generator=g, device="cuda")).to(dt)
    t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[::7] = -1
    dloss = torch.randn(T, generator=g, device="cuda") * most
    dloss[1::4] *= 2.0 ** -20
    dloss[2::4] *= 2.0 ** -34
    dloss[3::8] = 0.0
    loss, lse = ss.ss_linear_xent(h, w, t)
    got, want = ss.ss_linear_xent_bwd(dloss, h, w, t, lse), gradients(h, w, t, dloss)
    for k in ("dhidden", "dweight"):
        assert worst(got, want, k) <= 1.0, k
    assert not got["dhidden"][3::8].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_row_keeps_its_gradient_beside_a_larger_one(io):
    """The same token with and without a much larger dloss elsewhere in the batch: dhidden's row does not change."""
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(3)
    h, w = torch.randn(300, 64, generator=g, device="cuda").to(dt), (0.2 * torch.randn(5000, 64, generator=g, device="cuda")).to(dt)
    t = torch.arange(300, dtype=torch.int32, device="cuda")
    loss, lse = ss.ss_linear_xent(h, w, t)
    dloss = torch.full((300,), 2.0 ** -25, device="cuda")
    want = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)["dhidden"]
    dloss[0] = 1.0
    assert torch.equal(ss.ss_linear_xent_bwd(dloss, h, w, t, lse)["dhidden"][1:], want[1:])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [100, 500])
def test_one_dloss_for_all_and_zeros(io, T):
    """One power of two serves all rows then, and dweight takes the rows that the logits took."""
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(5)
    h, w = torch.randn(T, 200, generator=g, device="cuda").to(dt), (0.1 * torch.randn(3001, 200, generator=g, device="cuda")).to(dt)
    t = torch.randint(3001, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[::5] = -1
    loss, lse = ss.ss_linear_xent(h, w, t)
    for dloss in (torch.full((1,), 0.013, device="cuda").expand(T), torch.where(torch.arange(T, device="cuda") % 3 == 0, 0.0, -0.013)):
        got, want = ss.ss_linear_xent_bwd(dloss, h, w, t, lse), gradients(h, w, t, dloss)
        for k in ("dhidden", "dweight"):
            assert worst(got, want, k) <= 1.0, k


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_dloss_that_is_not_finite_stays_in_its_row(io, bad):
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(6)
    h, w = torch.randn(300, 64, generator=g, device="cuda").to(dt), (0.2 * torch.randn(900, 64, generator=g, device="cuda")).to(dt)
    t, dloss = torch.arange(300, dtype=torch.int32, device="cuda"), torch.randn(300, generator=g, device="cuda")
    loss, lse = ss.ss_linear_xent(h, w, t)
    dloss[7] = 0.0
    want = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)["dhidden"]
    dloss[7] = bad
    got = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)["dhidden"]
    keep = torch.arange(300) != 7
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[7]).any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_replayed_with_another_kind_of_dloss(io):
    """Captured while dloss is one value, replayed with values far apart, and back: what dweight takes follows the device's values."""
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(8)
    h, w = torch.randn(400, 96, generator=g, device="cuda").to(dt), (0.2 * torch.randn(1500, 96, generator=g, device="cuda")).to(dt)
    t = torch.randint(-1, 1500, (400,), generator=g, device="cuda", dtype=torch.int32)
    one = torch.full((400,), 0.25, device="cuda")
    apart = torch.exp2(-30 * torch.rand(400, generator=g, device="cuda"))
    loss, lse = ss.ss_linear_xent(h, w, t)
    want = [ss.ss_linear_xent_bwd(v, h, w, t, lse) for v in (one, apart)]
    dloss = one.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)
    for k in (0, 1, 1, 0):
        dloss.copy_((one, apart)[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got["dhidden"], want[k]["dhidden"]) and torch.equal(got["dweight"], want[k]["dweight"])
