"""The 8-bit norm where y is infinite but not NaN (weights that take it there): the block's scale is infinite, and by
y / scale its finite values are zeros and its infinite ones NaN; other blocks are untouched."""
import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [192, 200, 5000])
@pytest.mark.parametrize("block", [0, 32, 64])
def test_infinite_outputs(D, block):
    g = torch.Generator("cuda").manual_seed(D)
    x = 1.0 + torch.rand(3, D, generator=g, device="cuda")
    w = torch.ones(D, device="cuda")
    clean8, _, clean = ss.ss_add_rmsnorm_f8(x, w, block=block)
    w[70], w[D - 1] = float("inf"), float("-inf")
    y8, _, scale = ss.ss_add_rmsnorm_f8(x, w, block=block)
    got = y8.float()
    b = block or D
    for i in range(-(-D // b)):
        cols = slice(i * b, min(D, (i + 1) * b))
        if torch.isfinite(w[cols]).all():
            assert torch.equal(got[:, cols], clean8.float()[:, cols]) and torch.equal(scale[:, i], clean[:, i])
        else:
            assert (scale[:, i] == float("inf")).all()
            want = torch.where(torch.isinf(w[cols]), float("nan"), 0.0).expand(3, -1)
            assert torch.equal(torch.isnan(got[:, cols]), torch.isnan(want))
            assert not got[:, cols][~torch.isnan(want)].any()
