"""What is kept of weights far below the largest one, of which the header says 2^-28 of the largest, or 2^-39 where the
largest is below 2^-4 or 2^7 and above.  One row of the vocabulary has the large values, in columns that no other row has,
so that the other columns of dhidden come from the small rows alone: every element against the definition, off by
no more than that part of the largest weight times the sum of |dl|, besides the roundings of what is kept."""
import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from xent_bounds import gradients  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [60, 400])
@pytest.mark.parametrize("most,kept", [(2.0 ** -4, 2.0 ** -28), (1.0, 2.0 ** -32), (2.0 ** 6, 2.0 ** -38), (2.0 ** -5, 2.0 ** -39), (2.0 ** 7, 2.0 ** -39)])
@pytest.mark.parametrize("small", [2.0 ** -20, 2.0 ** -26])
def test_small_rows(io, T, most, kept, small):
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(T)
    h = (torch.randn(T, 64, generator=g, device="cuda") / max(most, 1.0)).to(dt)
    w = (most * small * torch.randn(700, 64, generator=g, device="cuda").clamp(-1, 1)).to(dt)
    w[:, :8] = 0
    w[5] = 0
    w[5, :8] = most
    t = torch.randint(700, (T,), generator=g, device="cuda", dtype=torch.int32)
    dloss = torch.randn(T, generator=g, device="cuda")
    loss, lse = ss.ss_linear_xent(h, w, t)
    got = ss.ss_linear_xent_bwd(dloss, h, w, t, lse)["dhidden"][:, 8:].double()
    want = gradients(h, w, t, dloss, w_kept=0.0)
    # |dl| of a row: at most 2 |dloss|
    bound = want["dhidden_bound"][:, 8:] + (kept * most * 2.0 * dloss.abs().double())[:, None]
    assert bool(((got - want["dhidden"][:, 8:]).abs() <= bound).all())
