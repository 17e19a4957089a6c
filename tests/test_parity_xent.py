"""Parity of the cross entropy over the vocabulary and its gradients with the 64-bit definition.

Tolerances.  A logit is a sum in fp32 of D products, taken 16 at a time; each of those D/16 additions may err by
2^-23 of the partial sum, which is at most |hidden| |weight| (the norms' product): loss and lse within
(D/16 + 16) 2^-23 of the largest such product, six times the additions in fp32 (three-part operands), and twice
that for the exponentials' and the logarithm's own roundings.  Gradients: fp32 relative L2 1e-5 (the scan's); in
bf16 dl is rounded to an operand and the result to its type, 2^-9 each on average over a step's halves: 5e-3."""
import ctypes

import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import training_ref as ref

from helpers import BF16_REL_L2, FP32_REL_L2, rel_l2, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


class Case:
    def __init__(self, T, V, D, io="bf16", ignored=0.2, seed=0, pad=0, scale=1.5):
        g = torch.Generator("cuda").manual_seed(seed + T + 3 * V + 7 * D)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
        self.T, self.V, self.D, self.io = T, V, D, io
        self.h = rn(T, D + pad).to(DT[io])[:, :D]
        self.w = (scale / D ** 0.5 * rn(V, D + pad)).to(DT[io])[:, :D]
        self.t = torch.randint(V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.t[torch.rand(T, generator=g, device="cuda") < ignored] = -1
        self.g = rn(T)

    def check(self, more=0.0):
        t = self.t.cpu().numpy().astype(np.int64)
        h, w, g = to_host(self.h), to_host(self.w), to_host(self.g)
        loss, lse = ss.ss_linear_xent(self.h, self.w, self.t)
        vl, vs = ref.xent(h, w, t)
        steps = self.D / 16 * (6 if self.io == "f32" else 1) + 16
        big = np.linalg.norm(h, axis=1) * np.linalg.norm(w, axis=1).max() + 1
        assert np.all(np.abs(to_host(lse) - vs) <= 2 * steps * 2.0 ** -23 * big), "lse"
        assert np.all(np.abs(to_host(loss) - vl) <= 2 * steps * 2.0 ** -23 * big), "loss"
        assert not loss[self.t < 0].any() and not lse[self.t < 0].any()
        d = ss.ss_linear_xent_bwd(self.g, self.h, self.w, self.t, lse)
        dh, dw = ref.xent_bwd(g, h, w, t)
        tol = more + (FP32_REL_L2 if self.io == "f32" else BF16_REL_L2)
        for k, v in (("dhidden", dh), ("dweight", dw)):
            assert d[k].dtype == DT[self.io] and rel_l2(to_host(d[k]), v) <= tol, f"{k}: {rel_l2(to_host(d[k]), v):.3e}"
        assert not d["dhidden"][self.t < 0].any()
        return loss, lse, d


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(64, 256, 64), (256, 256, 64), (256, 512, 256), (1, 2, 8), (3, 5, 7), (1, 1, 1), (45, 1000, 64), (257, 513, 130),
                                   (300, 4097, 768), (33, 9000, 1024), (700, 5003, 1111), (2, 300, 2560), (1500, 700, 96)])
def test_sizes(io, T, V, D):
    Case(T, V, D, io).check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(5000, 3000, 64), (4300, 9001, 72), (8192, 20000, 64)])
def test_many_rows(io, T, V, D):
    Case(T, V, D, io, ignored=0.4).check()


def test_pieces_of_the_vocabulary():
    """More columns than the workspace holds at once: the sums of dhidden grow from piece to piece."""
    Case(8192, 40000, 64, "bf16").check()
    Case(600, 140000, 64, "f32").check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 31, 64, 65, 127, 128, 129, 255])
def test_few_tokens(io, T):
    """About 128 tokens the shape of dhidden's product changes: both sides of it, sums in several slices of K."""
    Case(T, 9001, 320, io, ignored=0.0).check()
    Case(T, 9001, 320, io, ignored=0.5).check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_few_tokens_in_pieces_of_the_vocabulary(io):
    Case(20, 530000, 16, io).check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 8])
def test_strides(io, pad):
    c = Case(130, 700, 64, io, pad=pad)
    c.check()
    c.g = c.g[:1].expand(130)
    c.check()
    c.h = c.h[:1].expand(130, 64)
    c.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_targets(io):
    c = Case(520, 600, 64, io, ignored=0.0)
    c.check()
    c.t[:] = 599                                             # the same row of weight every time, in the last tile
    c.check()
    c.t[:256] = -1                                           # a whole tile of rows without
    c.check()
    c.t[:] = -5
    c.h[:] = NAN                                             # nothing is read
    loss, lse = ss.ss_linear_xent(c.h, c.w, c.t)
    d = ss.ss_linear_xent_bwd(c.g, c.h, c.w, c.t, lse)
    assert not loss.any() and not lse.any() and not d["dhidden"].any() and not d["dweight"].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_without_a_target_may_hold_anything(io):
    c = Case(300, 700, 96, io, ignored=0.5)
    want = c.check()
    off = c.t < 0
    c.h[off], c.g[off] = NAN, INF
    loss, lse = ss.ss_linear_xent(c.h, c.w, c.t)
    d = ss.ss_linear_xent_bwd(c.g, c.h, c.w, c.t, torch.where(off, NAN, lse))
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(d["dhidden"], want[2]["dhidden"]) and torch.equal(d["dweight"], want[2]["dweight"])


def test_targets_out_of_range_are_reported_and_left_out():
    c = Case(50, 300, 64, ignored=0.0)
    bad = c.t.clone()
    bad[3], bad[40], c.t[3], c.t[40] = 300, 2 ** 31 - 1, -1, -1
    got, want = ss.ss_linear_xent(c.h, c.w, bad), ss.ss_linear_xent(c.h, c.w, c.t)
    assert ss.device_error(clear=True) == 4
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = ss.ss_linear_xent_bwd(c.g, c.h, c.w, bad, got[1]), ss.ss_linear_xent_bwd(c.g, c.h, c.w, c.t, got[1])
    assert torch.equal(a["dhidden"], b["dhidden"]) and torch.equal(a["dweight"], b["dweight"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_non_finite_rows_stay_alone(io):
    c = Case(40, 300, 64, io, ignored=0.0)
    want = ss.ss_linear_xent(c.h, c.w, c.t)
    c.h[7, 3], c.h[20, 0] = NAN, INF
    loss, lse = ss.ss_linear_xent(c.h, c.w, c.t)
    keep = torch.ones(40, dtype=torch.bool)
    keep[[7, 20]] = False
    assert torch.equal(loss[keep], want[0][keep]) and torch.isnan(loss[7]) and not torch.isfinite(loss[20])
    d = ss.ss_linear_xent_bwd(c.g, c.h, c.w, c.t, lse)
    assert torch.isfinite(d["dhidden"][keep]).all() and torch.isnan(d["dhidden"][7]).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [40, 450])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -9, 1.5, 2.0 ** 9, 2.0 ** 60])
def test_magnitudes(io, T, scale):
    """Operands' scales follow the tensors' sizes: weight, hidden and dloss far from one, by the same pieces."""
    c = Case(T, 1500, 128, io)
    c.w, c.h = (c.w.double() * scale).to(DT[io]), (c.h.double() / max(scale, 1.0)).to(DT[io])
    c.check()
    c.g = c.g * scale
    c.check()
    c.g[::3] *= 2.0 ** -20                                   # weights of tokens far apart
    c.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_of_weight_of_unlike_sizes(io):
    """Rows of zeros (padding of the vocabulary), small ones and one that outweighs the others."""
    c = Case(450, 2000, 128, io)
    c.w[100:200] = 0
    c.w[200:300] *= 2.0 ** -30
    c.w[5] *= 8
    c.check()


def test_large_logits():
    """Logits of thousands: the exponentials neither overflow nor lose the row."""
    c = Case(100, 2000, 64, "f32", scale=800.0)
    c.check()


def test_sure_rows():
    """Rows whose target has nearly all of the probability: the gradient is the small difference p - 1 of the
    target's.  p = exp(l - lse) with both below 16: lse is stored with a half step of 2^-21, and the logit's sum errs
    by as much; the difference is off by 2^-20 at most, so the gradients, whose size is that of 1 - p, by
    2^-20 / (1 - p) of themselves."""
    c = Case(64, 500, 128, "f32", ignored=0.0)
    c.h = 8 * c.w[c.t.long()] / c.w[c.t.long()].norm(dim=1, keepdim=True)
    loss, lse = ref.xent(to_host(c.h), to_host(c.w), c.t.cpu().numpy())
    assert lse.max() < 16
    c.check(more=2.0 ** -20 / (1 - np.exp(-loss)).min())


def test_gradients_of_the_forward_call():
    """Directional differences of the losses themselves, in float32: a step of 2^-5 along a random direction."""
    c = Case(60, 400, 64, "f32")
    loss, lse = ss.ss_linear_xent(c.h, c.w, c.t)
    d = ss.ss_linear_xent_bwd(c.g, c.h, c.w, c.t, lse)
    f = lambda h, w: float((ss.ss_linear_xent(h, w, c.t)[0].double() * c.g).sum())          # noqa: E731
    torch.manual_seed(0)
    for k, at in (("dhidden", c.h), ("dweight", c.w)):
        v = torch.randn_like(at) * (at.norm() / at.numel() ** 0.5)
        s = 2.0 ** -5
        pair = [f(c.h + q * v, c.w) if k == "dhidden" else f(c.h, c.w + q * v) for q in (s, -s)]
        want = float((d[k].double() * v).sum())
        assert abs((pair[0] - pair[1]) / (2 * s) - want) <= 5e-3 * float((d[k].double().abs() * v.abs()).sum()), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_same_bits_every_time_and_scratch_of_any_contents(io):
    c = Case(700, 3000, 200, io)
    a = c.check()
    junk = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")   # what the next workspaces may hold
    del junk
    b = c.check()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


def test_no_tokens():
    c = Case(4, 300, 64)
    loss, lse = ss.ss_linear_xent(c.h[:0], c.w, c.t[:0])
    d = ss.ss_linear_xent_bwd(c.g[:0], c.h[:0], c.w, c.t[:0], lse)
    assert loss.shape == (0,) and d["dhidden"].shape == (0, 64) and not d["dweight"].any()


def test_outputs_with_strides_of_their_own():
    """Through the C ABI: rows of dhidden and dweight apart, the space between them left as it was."""
    for io in ("bf16", "f32"):
        c = Case(70, 330, 72, io)
        loss, lse = ss.ss_linear_xent(c.h, c.w, c.t)
        want = ss.ss_linear_xent_bwd(c.g, c.h, c.w, c.t, lse)
        for wide in (80, 75):
            dh = torch.full((70, wide), 7.0, dtype=DT[io], device="cuda")
            dw = torch.full((330, wide), 7.0, dtype=DT[io], device="cuda")
            s = ss.XentStrides(ss.SS_BF16 if io == "bf16" else ss.SS_F32, 72, 72, wide, wide, 1)
            n = ss.lib().ss_linear_xent_workspace_size(70, 330, 72, s.io_dtype, 1)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            st = ss.lib().ss_linear_xent_bwd(c.g.data_ptr(), c.h.data_ptr(), c.w.data_ptr(), c.t.data_ptr(), lse.data_ptr(), dh.data_ptr(),
                                             dw.data_ptr(), 70, 330, 72, ctypes.byref(s), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
            assert st == 0
            assert torch.equal(dh[:, :72], want["dhidden"]) and torch.equal(dw[:, :72], want["dweight"])
            assert (dh[:, 72:] == 7).all() and (dw[:, 72:] == 7).all()


def test_refusals():
    c = Case(10, 100, 64)
    loss, lse = ss.ss_linear_xent(c.h, c.w, c.t)
    with pytest.raises(TypeError):
        ss.ss_linear_xent(c.h, c.w.float(), c.t)
    with pytest.raises(TypeError):
        ss.ss_linear_xent(c.h, c.w, c.t.long())
    with pytest.raises(TypeError):
        ss.ss_linear_xent(c.h.half(), c.w.half(), c.t)
    with pytest.raises(ValueError):
        ss.ss_linear_xent(c.h, c.w[:, :63], c.t)
    with pytest.raises(ValueError):
        ss.ss_linear_xent(c.h, c.w, c.t[:9])
    with pytest.raises(ValueError):
        ss.ss_linear_xent(c.h.t(), c.w, c.t)
    with pytest.raises(ValueError):
        ss.ss_linear_xent_bwd(c.g[:9], c.h, c.w, c.t, lse)
    with pytest.raises(TypeError):
        ss.ss_linear_xent_bwd(c.g.double(), c.h, c.w, c.t, lse)
    with pytest.raises(ss.SelscanError):
        ss.ss_linear_xent(c.h, c.w[:1].expand(100, 64), c.t)             # rows of weight on top of each other
