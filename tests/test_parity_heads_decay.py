"""Single steps of a very strong decay among weak ones.  Such a token's own term outweighs all others' in the
outputs behind it, so that the errors of its factors do not average out; and the decays between the tokens
behind it are those of the weak steps, whatever the strong one's exponent.  Tolerances: those of the outputs and states
(bfloat16 outputs 5e-3 relative L2, over the tokens behind the step as over all; states 1e-5)."""
import pytest

import selective_state_space_scan_gb300 as ss

from helpers import BF16_REL_L2, FP32_REL_L2, STATE_REL_L2, rel_l2, to_host
from test_parity_heads import Case, Force

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


@pytest.mark.parametrize("io,path", [("bf16", 2), ("bf16", 1), ("f32", 1)])
@pytest.mark.parametrize("dt", [30.0, 1e3, 1e4, 1e5, 1e6, 1e30])
@pytest.mark.parametrize("at", [[0], [31], [32], [37], [64, 70], [128, 129, 130, 131], list(range(160, 190, 2))])
def test_strong_steps_among_weak_ones(io, path, dt, at):
    c = Case([260], H=4, N=64, io=io, seed=at[0] + len(at))
    c.dt_raw[at] = dt
    state, window = c.clone_caches()
    ry, rs, _ = c.reference(state, window)
    with Force(path=path):
        y = c.fwd(state, window)
    yh, sh = to_host(y), to_host(state)
    tol = BF16_REL_L2 if io == "bf16" else FP32_REL_L2
    assert rel_l2(yh, ry) <= tol, f"all: {rel_l2(yh, ry):.2e}"
    parts = [(at[-1] + 1, (at[-1] // 32 + 1) * 32), (at[-1] + 1, 260), (0, at[0])]
    for a, b in parts:
        if b > a:
            assert rel_l2(yh[a:b], ry[a:b]) <= tol, f"tokens {a} to {b}: {rel_l2(yh[a:b], ry[a:b]):.2e}"
    slot = int(c.slots[0])
    assert rel_l2(sh[slot], rs[slot]) <= STATE_REL_L2
