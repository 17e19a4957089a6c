"""The training calls in CUDA graphs, on several streams and from several threads: a call's workspace is its own."""
import threading

import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


class Work:
    """Inputs of every training call and the calls' results."""

    def __init__(self, seed, T=300, D=128, V=1000, io=torch.bfloat16):
        g = torch.Generator("cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
        self.x, self.dy, self.h = rn(T, D).to(io), rn(T, D).to(io), rn(T, D).to(io)
        self.res, self.dr, self.w, self.b = rn(T, D), rn(T, D), 1 + 0.1 * rn(D), rn(D)
        self.head = (rn(V, D) / D ** 0.5).to(io)
        self.t = torch.randint(-1, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.dloss = rn(T)
        self.c, self.dc, self.cw = rn(2, T, D).to(io), rn(2, T, D).to(io), rn(D, 4)
        self.logits = rn(T, V).to(io)
        self.ids = torch.randint(-1, V, (T, 9), generator=g, device="cuda", dtype=torch.int32)
        self.top = rn(T, 9)

    def run(self, stream=None):
        kw = dict(stream=stream)
        y, r, mean, rstd = ss.ss_add_layernorm(self.x, self.w, bias=self.b, residual=self.res, **kw)
        n = ss.ss_add_layernorm_bwd(self.dy, r, self.w, mean, rstd, dr=self.dr, **kw)
        c = ss.ss_conv1d_bwd(self.dc, self.c, self.cw, **kw)
        loss, lse = ss.ss_linear_xent(self.h, self.head, self.t, **kw)
        e = ss.ss_linear_xent_bwd(self.dloss, self.h, self.head, self.t, lse, **kw)
        kl, dl = ss.ss_distill_grad(self.dloss, self.logits, self.ids, self.top, **kw)
        kl2 = ss.ss_distill(self.logits, self.ids, self.top, **kw)
        return [y, r, mean, rstd, *n.values(), *[v for v in c.values() if v is not None], loss, lse, *e.values(), kl, dl, kl2]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed():
    works = [Work(s, io=io) for s, io in ((1, torch.bfloat16), (2, torch.float32))]
    want = [[t.clone() for t in w.run()] for w in works]
    graphs = []
    for w in works:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = w.run()
            again = w.run()                                  # (on memory that the first call's workspaces had)
        graphs.append((graph, out, again))
    torch.cuda.empty_cache()
    junk = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    for k in (1, 0, 0, 1):
        graph, out, again = graphs[k]
        for t in out + again:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want[k]) and same(again, want[k])
    del junk


def test_changed_inputs_reach_a_replay():
    w = Work(3)
    w.run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = w.run()
    other = Work(4)
    for k, v in vars(other).items():
        getattr(w, k).copy_(v)                               # (another number of rows with a target among them)
    graph.replay()
    torch.cuda.synchronize()
    assert same(out, other.run())


def test_streams_and_threads():
    works = [Work(s) for s in range(4)]
    want = [w.run() for w in works]
    torch.cuda.synchronize()
    got, bad = [None] * 4, []

    def call(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(5):
                if i % 2:
                    got[i] = works[i].run(stream)
                else:
                    with torch.cuda.stream(stream):
                        got[i] = works[i].run()
            stream.synchronize()
        except Exception as e:                               # noqa: BLE001
            bad.append(e)
    threads = [threading.Thread(target=call, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    torch.cuda.synchronize()
    for i in range(4):
        assert same(got[i], want[i])


def test_one_call_behind_another_on_the_same_tensors():
    """Back to back, without anything between: the second call's first kernel waits for the first call's last one."""
    w = Work(7)
    want = [t.clone() for t in w.run()]
    for _ in range(20):
        out = w.run()
    torch.cuda.synchronize()
    assert same(out, want)
