"""The serving calls at sizes at the ends of their ranges: rows of up to 2^19 logits, activations whose offsets
pass 32 bits, one long prompt among short ones, more counters than their part of the workspace holds,
and state counts that no vector kernel is made for."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import serving_ref as ref

from helpers import BF16_REL_L2, FP32_REL_L2, STATE_REL_L2, rel_l2, to_host
from test_parity_heads import IOS, Case, Force, check, run_fwd
from test_parity_sample import DT, noise_for
from test_parity_sample import check as check_tokens

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [131073, 262144, 300001, 524287, 524288])
def test_the_largest_vocabularies(io, V):
    g = torch.Generator("cuda").manual_seed(V)
    settings = [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.9, 40, 1.0, 0.0), (1.2, 0, 0.9, 0.0), (0.6, 500, 0.95, 0.02),
                (2.0, 60000, 0.97, 0.0), (100.0, 0, 0.5, 0.0), (1.0, V - 1, 0.3, 0.0)]
    rows = len(settings)
    t, k, p, m = (list(v) for v in zip(*settings))
    logits = (2.5 * torch.randn(rows, V, generator=g, device="cuda")).to(DT[io])
    check_tokens(logits, noise_for(rows, V, 1), t, k, p, m)
    same = torch.zeros(rows, V, device="cuda").to(DT[io])                  # every bin's sums at their largest
    same[:, ::3] = 1.0
    check_tokens(same, noise_for(rows, V, 2), t, k, p, m)


@pytest.mark.parametrize("path", [1, 2])
def test_activation_offsets_past_32_bits(path):
    """Sequences at the end of 120000 rows of 20000 elements: xbc, dt_raw, z and y all lie past 2^31 elements."""
    T, width, lens = 120000, 20000, [200, 131]
    c = Case(lens, H=2, N=64, seed=9)
    wide = torch.zeros(T, width, dtype=c.dt, device="cuda")
    out = torch.zeros(T, width, dtype=c.dt, device="cuda")
    HP, n = c.H * c.P, sum(lens)
    at = dict(z=slice(0, HP), xbc=slice(HP, HP + c.C), dt_raw=slice(HP + c.C, HP + c.C + c.H))
    for k, cols in at.items():
        wide[T - n:, cols] = getattr(c, k)
    state, window = c.clone_caches()
    want = c.reference(state, window)
    cu = torch.tensor([T - n, T - lens[1], T], dtype=torch.int32, device="cuda")
    with Force(path=path):
        y = ss.ss_heads_fwd(wide[:, at["xbc"]], wide[:, at["dt_raw"]], c.conv_w, c.A_log, state, window, cu, conv_b=c.conv_b,
                            dt_bias=c.dt_bias, D=c.D, z=wide[:, at["z"]], slots=c.slots, y=out[:, :HP])
    torch.cuda.synchronize()
    check(c, y[T - n:], state, window, want)
    assert not out[:T - n].any() and not out[:, HP:].any()


@pytest.mark.parametrize("io,path", [("bf16", 0), ("bf16", 2), ("f32", 0)])
def test_one_long_prompt_among_short_ones(io, path):
    with Force(path=path):
        run_fwd(Case([100, 100, 0, 12000, 100, 1, 90, 100], H=3, N=64, io=io, seed=10), f"{io} {path}")


@pytest.mark.parametrize("io", IOS)
def test_more_counters_than_their_part_of_the_workspace(io):
    """2100 requests of 8 groups: more than 16384 counters.  One token, then a prompt of two, then a token."""
    n, H, P, N = 2100, 8, 4, 8
    c = Case([1] * n, H=H, P=P, G=8, N=N, io=io, seed=11)
    d = Case([2] * n, H=H, P=P, G=8, N=N, io=io, seed=12)
    d.slots = c.slots
    state, window = c.clone_caches()
    for k in (c, d, c):
        want = k.reference(state, window)
        y = (k.step if k is c else k.fwd)(state, window)
        torch.cuda.synchronize()
        ry, rs, rw = want
        assert rel_l2(to_host(y), ry) <= (BF16_REL_L2 if io == "bf16" else FP32_REL_L2)
        assert rel_l2(to_host(state), rs) <= STATE_REL_L2
        np.testing.assert_array_equal(to_host(window), rw.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("N", [2, 17, 24, 40, 65, 96, 130, 192, 255, 256])
def test_steps_and_prompts_of_other_state_counts(io, N):
    c = Case([1] * 3, H=4, P=20, G=2, N=N, io=io, seed=N)
    state, window = c.clone_caches()
    for _ in range(2):
        want = c.reference(state, window)
        y = c.step(state, window)
        torch.cuda.synchronize()
        check(c, y, state, window, want, f"N={N}")
    run_fwd(Case([150, 3], H=4, P=20, G=2, N=N, io=io, seed=N), f"prompts N={N}")


def test_reference_sums_of_the_largest_rows():
    """(The definition's own running sums, in 64 bits, are exact enough at 2^19 equal weights.)"""
    l = np.zeros(1 << 19, np.float32)
    e = np.full(1 << 19, 2.0, np.float32)
    e[(1 << 18) - 1], e[1 << 18] = 1.0, 0.5
    assert ref.sample_row(l, e, top_p=0.5) == (1 << 18) - 1
