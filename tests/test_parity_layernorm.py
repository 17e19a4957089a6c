"""Parity of the residual layer norm and its backward pass with the 64-bit definitions.
Tolerances: float32 relative L2 2e-6 (a value takes at most 8 roundings of 2^-24 besides its sums, whose trees
of at most 64 + 10 additions in a row err by some 9 more on average); bfloat16 the half step of its rounding
beside that.  Sums over rows 2e-6 as well: at most 64 rows to a CTA and 32 CTAs to a warp in a row, with
rounding errors of either sign."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import training_ref as ref

from helpers import rel_l2, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2e-6


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def close(t, v, what, tol=F32):
    h = to_host(t)
    if t.dtype == torch.bfloat16:
        scale = np.sqrt(np.mean(v * v))
        assert np.all(np.abs(h - v) <= np.abs(v) * 2.0 ** -8 + 4 * tol * (np.abs(v) + scale)), what
    else:
        assert rel_l2(h, v) <= tol, f"{what}: {rel_l2(h, v):.3e}"


class Case:
    def __init__(self, rows, D, io="f32", res=None, pad=0, seed=0, bias=True, dr=True):
        g = torch.Generator("cuda").manual_seed(seed + 7 * D + rows)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
        self.rows, self.D = rows, D
        self.x = (0.3 + rn(rows, D + pad)).to(DT[io])[:, :D]
        self.res = None if res is None else (3 * rn(rows, D + pad)).to(DT[res])[:, :D]
        self.dy = rn(rows, D + pad).to(DT[io])[:, :D]
        self.dr = rn(rows, D + pad).to(DT[res or io])[:, :D] if dr else None
        self.w, self.b = 1 + 0.3 * rn(D), (0.2 * rn(D) if bias else None)

    def fwd(self, **kw):
        return ss.ss_add_layernorm(self.x, self.w, bias=self.b, residual=self.res, **kw)

    def check(self):
        h = lambda t: None if t is None else to_host(t)                  # noqa: E731
        y, r, mean, rstd = self.fwd()
        vy, vr, vm, vs = ref.layernorm(h(self.x), h(self.res), h(self.w), h(self.b), 1e-5)
        close(y, vy, "y")
        if self.res is None:
            assert r is self.x
        else:
            assert r.dtype == self.res.dtype
            close(r, vr, "residual")
        assert np.all(np.abs(h(mean) - vm) <= 2e-7 * np.sqrt((vr ** 2).mean(-1)) * 8)
        assert np.all(np.abs(h(rstd) - vs) <= F32 * vs)
        g = ss.ss_add_layernorm_bwd(self.dy, r, self.w, mean, rstd, dr=self.dr)
        d, dw, db = ref.layernorm_bwd(h(self.dy), h(r), h(self.w), h(mean), h(rstd), h(self.dr))
        assert g["dx"].dtype == self.dy.dtype and g["dresidual"].dtype == r.dtype
        for k, v in (("dx", d), ("dresidual", d), ("dweight", dw), ("dbias", db)):
            close(g[k], v, k)
        return y, r, mean, rstd, g


TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None), ("f32", None)]


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 2), (3, 7), (2, 64), (5, 100), (4, 768), (7, 2560), (3, 5120), (5, 4104), (2, 8191), (2, 8192),
                                    (3, 16384), (2, 16383), (700, 520), (2000, 1111)])
def test_types_and_sizes(io, res, rows, D):
    Case(rows, D, io, res).check()


def test_one_column():
    """A single column is its own mean: y is the bias, the gradient of x is that of r alone."""
    c = Case(5, 1, "f32", "f32")
    y, r, mean, rstd = c.fwd()
    g = ss.ss_add_layernorm_bwd(c.dy, r, c.w, mean, rstd, dr=c.dr)
    assert torch.equal(y, c.b.expand(5, 1)) and torch.equal(mean, r[:, 0]) and torch.equal(g["dx"], c.dr)
    assert not g["dweight"].any()


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("io,res", TYPES[:5])
def test_strides(io, res, pad):
    Case(9, 256, io, res, pad=pad).check()
    Case(300, 768, io, res, pad=pad, bias=False, dr=False).check()


def test_residual_in_place_and_broadcast_rows():
    c = Case(6, 320, "bf16", "f32")
    want = c.fwd()
    keep = c.res.clone()
    y, r, mean, rstd = ss.ss_add_layernorm(c.x, c.w, bias=c.b, residual=keep, residual_out=keep)
    assert r is keep and torch.equal(r, want[1]) and torch.equal(y, want[0]) and torch.equal(rstd, want[3])
    c.x, c.dy = c.x[:1].expand(6, 320), c.dy[:1].expand(6, 320)          # rows with a stride of zero
    c.check()


def test_far_from_zero():
    """A row of mean 1000 and deviation 1: its squares are taken about the mean.  (r - mean) has the mean's half
    step, 2^-25 · 1000, and so has r's own sum."""
    c = Case(64, 2560, "f32")
    c.x = c.x + 1000
    y, r, mean, rstd = c.fwd()
    vy, _, vm, vs = ref.layernorm(to_host(c.x), None, to_host(c.w), to_host(c.b), 1e-5)
    assert np.all(np.abs(to_host(rstd) - vs) <= F32 * vs)
    assert np.all(np.abs(to_host(mean) - vm) <= 1000 * 2.0 ** -22)
    assert rel_l2(to_host(y), vy) <= 1000 * 2.0 ** -22


def test_equal_rows_and_non_finite_rows():
    x = torch.full((4, 192), 2.5, device="cuda")
    w, b = torch.ones(192, device="cuda"), torch.full((192,), 0.25, device="cuda")
    x[1, 5], x[2, 100] = float("nan"), float("inf")
    y, r, mean, rstd = ss.ss_add_layernorm(x, w, bias=b)
    assert (y[0] == 0.25).all() and (y[3] == 0.25).all() and torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    dy = torch.ones(4, 192, device="cuda")
    g = ss.ss_add_layernorm_bwd(dy, r, w, mean, rstd)
    assert torch.isfinite(g["dx"][0]).all() and torch.isfinite(g["dx"][3]).all() and (g["dbias"] == 4).all()
    assert torch.isnan(g["dx"][1]).all() and torch.isnan(g["dweight"]).all()


def test_no_rows():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    y, r, mean, rstd = ss.ss_add_layernorm(e, w, residual=e)
    assert y.shape == (0, 64) and mean.shape == (0,)
    g = ss.ss_add_layernorm_bwd(e, e, w, mean, rstd)
    assert not g["dweight"].any() and not g["dbias"].any() and g["dx"].shape == (0, 64)


def test_same_bits_every_time():
    c = Case(5000, 768, "bf16", "f32")
    a, b = c.check()[4], c.check()[4]
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_rows_past_32_bit_offsets():
    rows, D = 300000, 8192                                   # 2.4e9 elements
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(D, device="cuda").to(torch.bfloat16)
    w = torch.ones(D, device="cuda")
    y, r, mean, rstd = ss.ss_add_layernorm(x, w)
    vy, _, vm, vs = ref.layernorm(to_host(x[-1:]), None, to_host(w), None, 1e-5)
    close(y[-1:], vy, "last row")
    assert not y[:-1:1000].any()
    dy = torch.zeros_like(x)
    dy[-1] = 1 + torch.arange(D, device="cuda").remainder(7)
    g = ss.ss_add_layernorm_bwd(dy, r, w, mean, rstd)
    d, dw, db = ref.layernorm_bwd(to_host(dy[-1:]), to_host(r[-1:]), to_host(w), to_host(mean[-1:]), to_host(rstd[-1:]))
    close(g["dx"][-1:], d, "last row's gradient")
    close(g["dweight"], dw, "dweight")
    close(g["dbias"], db, "dbias")


def test_refusals():
    c = Case(4, 64, "bf16", "f32")
    y, r, mean, rstd = c.fwd()
    with pytest.raises(ss.SelscanError):
        ss.ss_add_layernorm(c.x, c.w, residual=c.res, y=c.x)
    with pytest.raises(ss.SelscanError):
        ss.ss_add_layernorm(torch.zeros(1, 16385, device="cuda"), torch.ones(16385, device="cuda"))
    with pytest.raises(TypeError):
        ss.ss_add_layernorm(c.x.half(), c.w)
    with pytest.raises(ValueError):
        ss.ss_add_layernorm(c.x, c.w, bias=c.b[:63])
    with pytest.raises(ValueError):
        ss.ss_add_layernorm(c.x.t(), c.w)
    with pytest.raises(ValueError):
        ss.ss_add_layernorm_bwd(c.dy, r, c.w, mean[:3], rstd)
    with pytest.raises(TypeError):
        ss.ss_add_layernorm_bwd(c.dy, r, c.w, mean, rstd, dr=c.dr.bfloat16())
    with pytest.raises(ValueError):
        ss.ss_add_layernorm_bwd(c.dy, r[:3], c.w, mean, rstd)
