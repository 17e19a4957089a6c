"""cu_seqlens that decrease: a sequence that starts below an earlier entry is reported and skipped, on every
path, whatever the valid ranges would add up to; the others are what they are alone, and nothing is written
outside the workspace."""
import ctypes

import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import serving_ref as ref

from helpers import BF16_REL_L2, FP32_REL_L2, STATE_REL_L2, rel_l2, to_host
from test_parity_heads import Case, Force

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 1 << 20


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def valid(cu, T):
    top, ok = 0, []
    for a, b in zip(cu[:-1], cu[1:]):
        ok.append(0 <= a <= b <= T and a >= top)
        top = max(top, a)
    return ok


def run(cu, T, io, path=0, chunks=0, pre=0, H=3, N=48, seed=0):
    """One call through the C ABI on a workspace with a guard behind it, against the valid sequences."""
    n = len(cu) - 1
    c = Case([T], H=H, N=N, io=io, seed=seed, pool=n + 1)
    c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    c.slots = torch.randperm(n + 1, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32).cuda()
    state, window = c.clone_caches()
    y = torch.full((T, H * c.P), 7.0, dtype=c.dt, device="cuda")
    lib = ss.lib()
    with Force(path=path, chunks=chunks, pre=pre):
        code = ss.SS_BF16 if io == "bf16" else ss.SS_F32
        need = lib.ss_heads_workspace_size(n, T, H, c.P, c.G, N, code)
        ws = torch.zeros(need + GUARD, dtype=torch.uint8, device="cuda")
        ws[need:] = 0xA5
        s = ss.HeadsStrides(code, c.xbc.stride(0), c.dt_raw.stride(0), c.z.stride(0), y.stride(0))
        p = lambda t: t.data_ptr()                                       # noqa: E731
        assert lib.ss_heads_fwd(p(c.xbc), p(c.dt_raw), p(c.z), p(c.conv_w), p(c.conv_b), p(c.dt_bias), p(c.A_log), p(c.D), p(y),
                                p(state), p(window), p(c.cu), p(c.slots), None, n, T, H, c.P, c.G, N, n + 1, ctypes.byref(s),
                                p(ws), need, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
    ok = valid(cu, T)
    assert ss.device_error(clear=True) == (0 if all(ok) else 4)
    assert bool((ws[need:] == 0xA5).all())
    h = lambda t: to_host(t)                                             # noqa: E731
    yh, sh, wh = h(y), h(state), h(window)
    want_y, want_s, want_w = np.full(yh.shape, 7.0), h(c.state), h(c.window)
    par = [h(t) for t in (c.conv_w, c.conv_b, c.dt_bias, c.A_log, c.D)]
    xbc, dtr, z = h(c.xbc), h(c.dt_raw), h(c.z)
    for i, slot in enumerate(c.slots.tolist()):
        if ok[i]:
            r = slice(cu[i], cu[i + 1])
            want_y[r], want_s[slot], want_w[slot] = ref.heads(xbc[r], dtr[r], *par, z[r], want_s[slot], want_w[slot], c.P, N)
    assert rel_l2(yh, want_y) <= (BF16_REL_L2 if io == "bf16" else FP32_REL_L2)
    for k in range(n + 1):
        assert rel_l2(sh[k], want_s[k]) <= STATE_REL_L2, k
    np.testing.assert_array_equal(wh, want_w.astype(np.float32).astype(np.float64))


T = 1500
ORDERS = [[0, T, 0, T], [0, T, 0, T, 0, T, 0, T], [0, 700, 300, 900, 1200, T], [0, 10, 5, 5, 20, 4, T], [400, 900, 0, 400, T],
          [0, T, T, 0, 0, T], [0, T + 5, 3, T], [-1, 400, 900], [0, 300, 300, 1000, 999, T]]


@pytest.mark.parametrize("cu", ORDERS)
@pytest.mark.parametrize("io,force", [("bf16", dict(path=2, chunks=-1)), ("bf16", dict(path=2, chunks=-4)),
                                      ("bf16", dict(path=2, chunks=2)), ("bf16", dict(path=2)), ("f32", dict(path=1, pre=1)),
                                      ("f32", dict(path=1, pre=2)), ("bf16", dict(path=1))])
def test_decreasing_entries(io, force, cu):
    run(cu, T, io, seed=len(cu), **force)


@pytest.mark.parametrize("force", [dict(path=2, chunks=-1), dict(path=2, chunks=3), dict(path=1, pre=2), dict(path=1, pre=1)])
def test_a_late_fault_among_many_sequences(force):
    """Hundreds of sequences, more than one block looks at in one go: the fault is in the last ones."""
    cu = [2 * i for i in range(600)]
    cu[577], cu[590] = 3, 1000                                           # (sequences 577 and 590: below and decreasing)
    run(cu, cu[-1], "bf16", H=1, N=32, seed=3, **force)


def test_short_sequences_and_whole_passes():
    for io in ("bf16", "f32"):
        run([0, 20, 10, 30, 25, 40], 40, io, seed=1)
        run([0, 0, 0, 40, 0, 40], 40, io, path=1, pre=1, H=40, seed=2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 255, 256, 1100])
def test_faults_among_many_short_sequences(io, n):
    """Sequences of a token or two, many of them out of order, around the number from which one launch looks at
    their order for all, and past what that looks at in one go."""
    rng = np.random.default_rng(n)
    cu = np.concatenate([[0], np.cumsum(rng.integers(0, 3, n))]).tolist()
    T = cu[-1]
    for i in rng.choice(n, 9, replace=False).tolist() + [n - 1]:
        cu[i] = int(rng.integers(-1, T + 2))
    run(cu, T, io, path=1, pre=1, H=9 if n < 100 else 40, N=16, seed=n)
