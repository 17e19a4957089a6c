"""The two tiles that a CTA of the products' path works on share one set of scores C·Bᵀ: neither may get the
next chunk's before it has read its own.  Here one of them is held up (channels that are not finite take the
long way), which has to change nothing in the other."""
import pytest

import selective_state_space_scan_gb300 as ss

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


def run(c):
    state, window = c.clone_caches()
    y = c.fwd(state, window)
    torch.cuda.synchronize()
    return y, state


@pytest.mark.parametrize("slow", [0, 1])
@pytest.mark.parametrize("chunks", [0, -1, -3, 4])
def test_a_slow_tile_changes_nothing_in_the_other(chunks, slow):
    c = Case([1700, 129, 640, 0, 3000], H=8, N=128, seed=80 + slow)
    with Force(path=2, chunks=chunks):
        y0, s0 = run(c)
        for h in range(slow, c.H, 2):                          # every second head, every second channel of it
            c.xbc[:, h * c.P + 1:(h + 1) * c.P:2] = float("inf")
        for _ in range(5):
            y1, s1 = run(c)
            for h in range(1 - slow, c.H, 2):
                r = slice(h * c.P, (h + 1) * c.P)
                assert torch.equal(y0[:, r], y1[:, r])
                assert torch.equal(s0[:, h], s1[:, h])


def test_repeats_over_many_pieces_are_bitwise_equal():
    """CTAs with many pieces one after the other, an odd tile without a neighbour among them."""
    c = Case([900, 260, 1, 1500, 128, 77, 640], H=33, N=64, seed=90)
    with Force(path=2, chunks=-2):
        first = run(c)
        for _ in range(10):
            again = run(c)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
