"""Threads that call on one stream: a call that passes data from launch to launch through the stream's
workspace has to put all of them on the stream before another thread's begins, and nobody may replace the
workspace in between.  No GPU: the library is a stand-in that counts the callers inside it."""
import threading
import time
from types import SimpleNamespace

import pytest

import selective_state_space_scan_gb300 as ss
from selective_state_space_scan_gb300 import serving

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on device 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class Library:
    """Every call takes a while; how many are inside at once, by stream."""

    def __init__(self, meet=None):
        self.inside, self.most, self.guard, self.meet = {}, 0, threading.Lock(), meet

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 4096
        if name == "ss__capture_id":
            return lambda handle: 0
        if name == "ss_status_string":
            return lambda code: b"an error"
        return self.call

    def call(self, *args):
        stream = args[-1]
        with self.guard:
            self.inside[stream] = self.inside.get(stream, 0) + 1
            self.most = max(self.most, self.inside[stream])
        if self.meet is not None:
            self.meet.wait(10)
        time.sleep(0.002)
        with self.guard:
            self.inside[stream] -= 1
        return 0


@pytest.fixture
def library(monkeypatch):
    serving._load()
    library = Library()
    monkeypatch.setattr(ss, "lib", lambda: library)
    monkeypatch.setattr(serving, "_lib", library)
    monkeypatch.setattr(ss, "workspace_for", lambda device, stream, nbytes, purpose="fwd": torch.zeros(nbytes, dtype=torch.uint8))
    for name, module in (("_HEADS_WS", serving), ("_HEADS_BYTES", serving), ("_WS_SIZES", ss)):
        if hasattr(module, name):
            monkeypatch.setattr(module, name, {})
    return library


def dev(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def heads(stream, call):
    H, P, N, T = 2, 8, 4, 3
    C = H * P + 2 * N
    state, window, y = dev(T, H, P, N), dev(T, C, 3), dev(T, H * P)
    a = (dev(T, C), dev(T, H), dev(C, 4), dev(H))
    if call == "step":
        return ss.ss_heads_step(state, window, *a, y=y, stream=stream)
    return ss.ss_heads_fwd(*a, state, window, dev(2, dtype=torch.int32), y=y, stream=stream)


def scan(stream, call):
    b, L, D, N = 1, 4, 8, 16
    t = torch.zeros
    a = (t(b, L, D), t(b, L, D), t(D), t(D, N), t(b, L, N), t(b, L, N))
    if call == "fwd":
        return ss.ss_fwd(*a, stream=stream, workspace=True)
    if call == "ckpt":
        return ss.ss_fwd_ckpt(*a, stream=stream)
    return ss.ss_bwd(t(b, L, D), *a, stream=stream)


CALLS = [(heads, "fwd"), (heads, "step"), (scan, "fwd"), (scan, "ckpt"), (scan, "bwd")]


def in_threads(jobs):
    errors = []

    def work(job):
        try:
            job()
        except BaseException as e:                            # noqa: BLE001 (shown by the assertion below)
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert not errors and not any(t.is_alive() for t in threads), errors


@pytest.mark.parametrize("f,call", CALLS)
def test_calls_on_one_stream_follow_one_another(library, f, call):
    stream = SimpleNamespace(cuda_stream=77, device=torch.device("cpu"))
    in_threads([lambda: [f(stream, call) for _ in range(5)]] * 4)
    assert library.most == 1


@pytest.mark.parametrize("f,call", CALLS)
def test_calls_on_two_streams_do_not_wait_for_each_other(library, f, call):
    library.meet = threading.Barrier(2)                        # (passed only with both inside)
    in_threads([lambda k=k: f(SimpleNamespace(cuda_stream=100 + k, device=torch.device("cpu")), call) for k in range(2)])


def test_an_error_frees_the_stream(library, monkeypatch):
    stream = SimpleNamespace(cuda_stream=78, device=torch.device("cpu"))
    monkeypatch.setattr(Library, "call", lambda self, *a: 1)

    def job():
        for f, call in CALLS:
            with pytest.raises(ss.SelscanError):
                f(stream, call)
    in_threads([job, job])
