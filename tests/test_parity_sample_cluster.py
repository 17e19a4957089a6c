"""The sampler's rows that a cluster of CTAs shares, where some of them have little or nothing to do: the last
slice empty or a single token, the few largest logits in one slice, and many rows at once.  A small top_k
stores to the shared memory of the cluster's other CTAs, which have to have begun by then."""
import pytest

import selective_state_space_scan_gb300 as ss

from test_parity_sample import DT, check, noise_for

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


# tokens of a slice are (V / CTAs) rounded up to 8: with 8 CTAs the last has V - 7 * that many
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4096, 8192, 16384 + 1, 32768 + 7, 32776, 16385 * 3, 65537])
def test_small_top_k_over_uneven_slices(io, V):
    g = torch.Generator("cuda").manual_seed(V)
    rows = 3
    l = (2 * torch.randn(rows, V, generator=g, device="cuda")).to(DT[io])
    l[0, -3:] = 20.0                                            # the leaders in the last slice
    l[1, :3] = 20.0                                             # and in the first
    for k in (1, 2, 3, 17, 128, 500):
        check(l, noise_for(rows, V, k), [0.9] * rows, [k] * rows, [1.0, 0.9, 0.5], [0.0] * rows)


def test_many_clusters_with_a_small_top_k():
    """More clusters than run at once, so that CTAs of a cluster begin while others end; the same tokens
    every time."""
    rows, V = 456, 16384
    g = torch.Generator("cuda").manual_seed(2)
    l = 2 * torch.randn(rows, V, generator=g, device="cuda")
    e = noise_for(rows, V)
    k = torch.randint(1, 100, (rows,), generator=g, device="cuda").to(torch.int32)
    first = ss.ss_sample(l, e, top_k=k)
    larger = (l > l.gather(1, first.long()[:, None])).sum(1)
    assert bool((larger < k).all())
    for _ in range(10):
        assert torch.equal(first, ss.ss_sample(l, e, top_k=k))
