"""Calls captured in CUDA graphs: a graph is whole by itself.  The workspace of a captured call has its
zeros from a node of the same graph, whatever its memory holds when the graph is launched, whichever of
several graphs runs first, and whatever becomes of the buffers that calls outside of graphs use."""
import pytest

import selective_state_space_scan_gb300 as ss

from helpers import rel_l2, to_host
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


class Captured:
    """A call on caches of its own, captured as `times` calls in a row (and run before that on another stream, as
    its kernels have to be loaded)."""

    def __init__(self, c, call, times=1, **kw):
        self.c, self.call, self.times = c, call, times
        getattr(c, call)(*c.clone_caches())
        self.state, self.window = c.clone_caches()
        self.graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(self.graph, **kw):
            for _ in range(times):
                self.y = getattr(c, call)(self.state, self.window)

    def check(self):
        """One launch from the starting caches against the same calls outside of a graph: bit for bit."""
        self.state.copy_(self.c.state)
        self.window.copy_(self.c.window)
        self.graph.replay()
        state, window = self.c.clone_caches()
        for _ in range(self.times):
            y = getattr(self.c, self.call)(state, window)
        torch.cuda.synchronize()
        assert torch.equal(self.window, window)
        assert torch.equal(self.state, state) and torch.equal(self.y, y)


def new_buffers(before):
    """Workspaces that the binding has made since."""
    held = list(ss._WORKSPACES.values()) + [w for _, w in getattr(ss, "_CAPTURED", {}).values()]
    return [w for w in held if all(w is not b for b in before)]


def test_the_second_graph_first():
    for c in (Case([1], seed=1), Case([40], io="f32", G=2, seed=3)):       # (the default stream's own buffer)
        c.fwd(*c.clone_caches())
    before = list(ss._WORKSPACES.values())
    one = Captured(Case([1] * 4, io="bf16", seed=1), "step", times=2)
    two = Captured(Case([1] * 2, io="bf16", seed=2), "step", times=2)
    three = Captured(Case([7, 20], io="f32", G=2, seed=3), "fwd")
    torch.cuda.synchronize()
    for w in new_buffers(before):                            # what memory that no graph has cleared may hold
        w.fill_(255)
    for g in (two, three, one, two):
        g.check()


def test_graphs_outlive_other_buffers():
    """Calls outside of graphs before the capture, on the same stream, and larger ones after it, whose
    workspace replaces the first; the graph still has its own memory."""
    side = torch.cuda.Stream()
    small = Case([1] * 3, io="bf16", seed=4)
    with torch.cuda.stream(side):
        small.step(*small.clone_caches())
    torch.cuda.synchronize()
    graphs = [Captured(small, "step", stream=side), Captured(Case([300, 90], seed=5), "fwd", stream=side),
              Captured(Case([900], io="f32", seed=6), "fwd", stream=side)]
    with torch.cuda.stream(side):
        large = Case([2000, 1000, 500], H=16, seed=7)
        large.fwd(*large.clone_caches())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    for g in graphs + graphs:
        g.check()
    del junk


def test_scan_with_a_workspace_in_two_graphs():
    """The older calls' workspaces (the balanced schedule's flags, the time split's states) in the same way."""
    torch.manual_seed(0)
    before = list(ss._WORKSPACES.values())
    made = []
    for batch, L, Dm in ((8, 256, 512), (1, 4096, 64)):
        t = lambda *s: torch.randn(*s, device="cuda")                     # noqa: E731
        a = (t(batch, L, Dm), t(batch, L, Dm) - 3, t(Dm), torch.log(1 + 15 * torch.rand(Dm, 16, device="cuda")),
             t(batch, L, 16), t(batch, L, 16), t(Dm), t(batch, L, Dm))
        last = torch.empty(batch, Dm, 16, device="cuda")
        ss.ss_fwd(*a, last_state=last, workspace=True)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            y = ss.ss_fwd(*a, last_state=last, workspace=True)
        made.append((g, a, y, last))
    torch.cuda.synchronize()
    for w in new_buffers(before):
        w.fill_(0xFF)
    for g, a, y, last in made[::-1] + made:
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        want_last = torch.empty_like(last)
        want = ss.ss_fwd(*a, last_state=want_last)
        assert rel_l2(to_host(y), to_host(want)) <= 1e-5 and rel_l2(to_host(last), to_host(want_last)) <= 1e-5
