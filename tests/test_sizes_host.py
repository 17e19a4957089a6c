"""The binding remembers workspace sizes: a bounded number of them, each for its device.  No GPU: the library is
a stand-in."""
from types import SimpleNamespace

import pytest

import selective_state_space_scan_gb300 as ss
from selective_state_space_scan_gb300 import serving

from test_threads_host import OnDevice, dev, library  # noqa: F401 (a fixture)

torch = pytest.importorskip("torch")

STREAM = SimpleNamespace(cuda_stream=5, device=torch.device("cpu"))


class OnDevice1(OnDevice):
    def get_device(self):
        return 1


def prompt(T, as_class=OnDevice):
    H, P, N = 1, 8, 4
    C = H * P + 2 * N
    t = lambda *s, **k: dev(*s, **k).as_subclass(as_class)                 # noqa: E731
    return ss.ss_heads_fwd(t(T, C), t(T, H), t(C, 4), t(H), t(2, H, P, N), t(2, C, 3), t(2, dtype=torch.int32), y=t(T, H * P),
                           stream=STREAM)


def test_prompts_of_every_length_do_not_fill_the_memory(library):            # noqa: F811
    for T in range(1, 3001):
        prompt(T)
    assert len(serving._HEADS_BYTES) <= 1024
    for L in range(1, 3001):
        ss.ss_fwd_workspace_size(1, L, 8, 16)
    assert len(ss._WS_SIZES) <= 1024


def test_a_size_is_that_of_its_device(library, monkeypatch):                 # noqa: F811
    """The plan depends on the device's SM count: a size asked for on one is not used on another."""
    asked, sizes = [], {0: 4096, 1: 8192}
    at = {"device": 0}

    def size(*key):
        asked.append(at["device"])
        return sizes[at["device"]]

    passed = []
    monkeypatch.setattr(type(library), "ss_heads_workspace_size", staticmethod(size), raising=False)
    monkeypatch.setattr(type(library), "ss_heads_fwd", staticmethod(lambda *a: passed.append(a[-2]) or 0), raising=False)
    for d, kind in ((0, OnDevice), (1, OnDevice1), (0, OnDevice), (1, OnDevice1)):
        at["device"] = d
        prompt(7, kind)
    assert asked == [0, 1] and passed == [4096, 8192, 4096, 8192]
