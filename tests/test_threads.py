"""Two threads that call on one stream at the same time get what each gets alone."""
import threading

import pytest

import selective_state_space_scan_gb300 as ss

from test_parity_heads import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def test_threads_on_one_stream():
    cases = [(Case([300, 90, 500], seed=1), "fwd"), (Case([1200], H=6, seed=2), "fwd"), (Case([900, 20], io="f32", seed=3), "fwd"),
             (Case([1] * 5, seed=4), "step")]

    def once(c, call):
        state, window = c.clone_caches()
        return getattr(c, call)(state, window), state, window

    want = [once(*k) for k in cases]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = [[] for _ in cases]
    start = threading.Barrier(len(cases))

    def work(i):
        with torch.cuda.stream(stream):
            start.wait(30)
            for _ in range(20):
                got[i].append(once(*cases[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    for w, results in zip(want, got):
        assert len(results) == 20
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(w, r))
