"""Long sequences of the token-by-token scan, which are cut in segments: the first pass leaves what every
segment but the last leaves, and puts the starting state in the last one's place.  B and C come
convolved by bulk copies; the last segment's CTA of that pass ends at once and must issue none."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss

from test_parity_heads import Case, Force, run_fwd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


@pytest.mark.parametrize("fresh", [[0, 0, 0, 0], [1, 1, 1, 1], [0, 1, 1, 0]])
@pytest.mark.parametrize("pre", [1, 2])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 64, 128])
def test_cut_sequences_fresh_and_warm(io, N, pre, fresh):
    c = Case([2100, 40, 0, 1333], H=2, N=N, io=io, seed=N + pre)
    c.fresh = torch.tensor(fresh, dtype=torch.int32, device="cuda")
    with Force(path=1, pre=pre):
        first = run_fwd(c, f"{io} N={N} pre={pre} {fresh}")
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, run_fwd_only(c)))


def run_fwd_only(c):
    state, window = c.clone_caches()
    y = c.fwd(state, window)
    torch.cuda.synchronize()
    return y, state, window


def test_blocks_that_follow_an_early_exit():
    """Many heads, so that other blocks take the place of those that end early: no value of theirs changes
    over repeats, and every head is what it is alone."""
    c = Case([3000], H=40, N=128, io="f32", seed=5)
    with Force(path=1, pre=2):
        first = run_fwd_only(c)
        assert np.isfinite(first[0].cpu().numpy()).all()
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(first, run_fwd_only(c)))
        one = Case([3000], H=1, N=128, io="f32", seed=6)
        one.xbc = torch.cat([c.xbc[:, :64], c.xbc[:, 40 * 64:]], 1)
        one.dt_raw, one.z = c.dt_raw[:, :1], c.z[:, :64]
        keep = torch.cat([torch.arange(64), torch.arange(40 * 64, c.C)]).cuda()
        one.conv_w, one.conv_b = c.conv_w[keep].contiguous(), c.conv_b[keep].contiguous()
        one.dt_bias, one.A_log, one.D = c.dt_bias[:1], c.A_log[:1], c.D[:1]
        one.state, one.window = c.state[:, :1].contiguous(), c.window[:, keep].contiguous()
        one.slots = c.slots
        y, state, window = run_fwd(one, "one head")
        assert float((y - first[0][:, :64]).norm() / y.norm()) <= 1e-5
